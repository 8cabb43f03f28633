"""The operators around a MoLE layer in a training step, as a program calls them,
and their plain forms: the embedding lookup and its gradient, the norms before
and after a block with its gate and residual scale, and the AdamW step.

    embed       out[t] = scale E[ids[t]]
    embed_grad  dE[ids[t]] += scale dout[t]                        (fp32, in place)
    norm        y = f / rms(f) w_post;  x' = res_scale x + gate y;  h = x' / rms(x') w_pre
    norm_grad   its backward pass: dx, df, dgate, and dw_pre, dw_post added to
    adamw       one step over a list of tensors, states in 32 or in 8 bits

`own` false: elementary torch operations in fp32, rounded once at the end.
`own` true: the framework's calls.
"""
import math

import torch

own = False

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
EPS = 1e-6
BLOCK = 128          # elements per scale of an 8-bit state
E4M3_MAX = 448.0
ADAM = dict(lr=1e-4, beta1=0.9, beta2=0.95, eps=1e-8, step=7)


def listed():
    return [
        # one decode step of 8 sequences: the lookup is all launch latency
        dict(name="embed-step", op="embed", T=8, D=2048, V=50304, table="bf16", out="bf16", ids="zipf"),
        # a prefill batch of the 1B shape into an fp32 residual stream
        dict(name="embed-prompt", op="embed", T=16384, D=2048, V=50304, table="bf16", out="f32", ids="zipf"),
        # a short ragged batch of an odd-width model
        dict(name="embed-grad-ragged", op="embed_grad", T=777, D=1001, V=50304, dout="bf16", ids="zipf"),
        # a training batch of text at the 1B shape: one id in seven tokens
        dict(name="embed-grad-text", op="embed_grad", T=16384, D=2048, V=50304, dout="f32", ids="zipf"),
        # a large batch whose ids hardly repeat: the gradient rows are the traffic
        dict(name="embed-grad-uniform", op="embed_grad", T=65536, D=1024, V=50304, dout="bf16", ids="uniform"),
        # one decode step of 8 sequences between two blocks
        dict(name="norm-step", op="norm", T=8, D=2048, x="f32", f="f32", h="bf16", gate=False),
        # a prefill batch of the 1B shape
        dict(name="norm-prompt", op="norm", T=16384, D=2048, x="f32", f="f32", h="bf16", gate=True),
        # a short ragged batch of an odd-width model with a bf16 stream
        dict(name="norm-grad-ragged", op="norm_grad", T=1237, D=1001, x="bf16", f="bf16", gate=True),
        # a training batch of the 1B shape
        dict(name="norm-grad-batch", op="norm_grad", T=16384, D=2048, x="f32", f="f32", gate=True),
        # routers and norm weights of 24 layers: many small tensors, odd sizes
        dict(name="adamw-small", op="adamw", tensors=72, mean=6000, largest=16384, param="f32", grad="f32", state=32),
        # one layer's experts, the embedding and the small weights of the 410M shape
        dict(name="adamw-layer", op="adamw", tensors=6, mean=2048, largest=67108864, param="master", grad="f32", state=32),
        # the same with 8-bit states
        dict(name="adamw-layer-8bit", op="adamw", tensors=6, mean=2048, largest=67108864, param="master", grad="f32",
             state=8),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["embed", "embed_grad", "norm", "norm_grad", "adamw"])
    if op == "adamw":
        return dict(op=op, tensors=rng.randint(1, 90), mean=_log(rng, 300, 200000), largest=_log(rng, 5000, 60000000),
                    param=rng.choice(["f32", "master", "bf16"]), grad=rng.choice(["f32", "bf16"]),
                    state=rng.choice([32, 8]))
    D = _log(rng, 64, 4096)
    if rng.random() < 0.6:
        D = (D + 7) // 8 * 8
    T = min(_log(rng, 1, 65536), (1 << 25) // D)
    if op == "embed":
        return dict(op=op, T=T, D=D, V=_log(rng, 512, 60000), table=rng.choice(["f32", "bf16"]),
                    out=rng.choice(["f32", "bf16"]), ids=rng.choice(["zipf", "uniform"]))
    if op == "embed_grad":
        return dict(op=op, T=T, D=D, V=_log(rng, 512, 50000), dout=rng.choice(["f32", "bf16"]),
                    ids=rng.choice(["zipf", "uniform"]))
    case = dict(op=op, T=T, D=D, x=rng.choice(["f32", "bf16"]), f=rng.choice(["f32", "bf16"]), gate=rng.random() < 0.5)
    if op == "norm":
        case["h"] = rng.choice(["f32", "bf16"])
    return case


def _distinct(T, V, kind):
    """Expected distinct ids of a batch."""
    if kind == "uniform":
        return V * -math.expm1(T * math.log1p(-1.0 / V))
    k = torch.arange(1, V + 1, dtype=torch.float64)
    p = k ** -1.1
    p /= p.sum()
    return float((-torch.expm1(T * torch.log1p(-p))).sum())


def _sizes(case):
    """Element counts of the optimizer's tensors: the large ones (two of the
    largest size, one of about three quarters of it), then small ones spread
    around the mean, odd counts among them."""
    big = [case["largest"], case["largest"], case["largest"] * 3 // 4][:max(1, case["tensors"] // 2)]
    small = [max(1, case["mean"] * (1 + (7 * i) % 11) // 6 + i % 3) for i in range(case["tensors"] - len(big))]
    return big + small


def work(case):
    op = case["op"]
    if op == "adamw":
        n = sum(_sizes(case))
        grad = 4 if case["grad"] == "f32" else 2
        param = {"f32": 8, "master": 10, "bf16": 4}[case["param"]]
        state = 16 if case["state"] == 32 else 4 + 16 / BLOCK
        return {"bytes": n * (grad + param + state), "flops": 16 * n}
    size = {"f32": 4, "bf16": 2}
    T, D = case["T"], case["D"]
    if op == "embed":
        U = _distinct(T, case["V"], case["ids"])
        return {"bytes": 4 * T + U * D * size[case["table"]] + T * D * size[case["out"]], "flops": T * D}
    if op == "embed_grad":
        U = _distinct(T, case["V"], case["ids"])
        return {"bytes": 4 * T + T * D * size[case["dout"]] + 8 * U * D, "flops": 2 * T * D}
    gate = 4 * T if case["gate"] else 0
    if op == "norm":
        return {"bytes": T * D * (2 * size[case["x"]] + size[case["f"]] + size[case["h"]]) + 8 * D + gate,
                "flops": 10 * T * D}
    return {"bytes": T * D * (size[case["x"]] + size[case["f"]] + 4 * 4) + 24 * D + 2 * gate, "flops": 24 * T * D}


def _ids(case, gen):
    T, V = case["T"], case["V"]
    if case["ids"] == "uniform":
        return torch.randint(0, V, (T,), generator=gen, device="cuda", dtype=torch.int32)
    cdf = torch.cumsum(torch.arange(1, V + 1, device="cuda", dtype=torch.float64) ** -1.1, 0)
    u = torch.rand(T, generator=gen, device="cuda", dtype=torch.float64) * cdf[-1]
    return torch.searchsorted(cdf, u, right=True).clamp_(max=V - 1).to(torch.int32)


def _encode(x):
    """Blocks of 128 fp32 values as e4m3 codes and fp32 scales."""
    b = x.view(-1, BLOCK)
    scale = (b.abs().amax(1) * (1.0 / E4M3_MAX)).clamp_min(2.0 ** -120)
    return (b * scale.reciprocal()[:, None]).to(torch.float8_e4m3fn).view(-1), scale


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)

    def normal(*shape, std=1.0, dtype=torch.float32):
        return torch.randn(shape, generator=gen, device="cuda").mul_(std).to(dtype)

    op = case["op"]
    s = {"case": case}
    if op == "embed":
        s["ids"] = _ids(case, gen)
        s["E"] = normal(case["V"], case["D"], std=0.02, dtype=TYPES[case["table"]])
        s["scale"] = math.sqrt(case["D"])
    elif op == "embed_grad":
        s["ids"] = _ids(case, gen)
        s["dout"] = normal(case["T"], case["D"], dtype=TYPES[case["dout"]])
        s["dE"] = normal(case["V"], case["D"])  # what the layers have added so far
        s["scale"] = math.sqrt(case["D"])
    elif op in ("norm", "norm_grad"):
        T, D = case["T"], case["D"]
        s["f"] = normal(T, D, std=0.3, dtype=TYPES[case["f"]])
        s["x"] = normal(T, D, std=2.0, dtype=TYPES[case["x"]])  # norm_grad: the forward's x'
        s["w_pre"], s["w_post"] = normal(D, std=0.1) + 1, normal(D, std=0.1) + 0.5
        s["gate"] = torch.sigmoid(normal(T)) if case["gate"] else None
        s["res_scale"] = 0.8
        if op == "norm_grad":
            s["dx_out"], s["dh"] = normal(T, D), normal(T, D)
            s["dw_pre"], s["dw_post"] = normal(D), normal(D)
    else:
        # every tensor starts on a block of its own in one flat buffer per kind;
        # a program's tensors are the views
        sizes = _sizes(case)
        at = [0]
        for n in sizes:
            at.append(at[-1] + (n + BLOCK - 1) // BLOCK * BLOCK)
        used = torch.zeros(at[-1], dtype=torch.bool, device="cuda")
        for a, n in zip(at, sizes):
            used[a:a + n] = True
        p, m = normal(at[-1], std=0.02), normal(at[-1], std=1e-3)
        root = normal(at[-1], std=2e-3).abs_()  # sqrt(v)
        g = normal(at[-1], std=2e-3)
        for buf in (p, m, root, g):
            buf.mul_(used)
        s["grad"] = g.to(TYPES[case["grad"]])
        s["param"] = p if case["param"] == "f32" else p.to(torch.bfloat16)
        s["master"] = p if case["param"] == "master" else None
        if case["state"] == 32:
            s["m"], s["v"] = m, root.square_()
        else:
            (s["m"], s["m_scale"]), (s["v"], s["v_scale"]) = _encode(m), _encode(root)
        # weights decay, the small tensors (norms, routers) do not
        s["decay"] = [0.1 if n > 4 * case["mean"] else 0.0 for n in sizes]
        blocks = torch.tensor([(b - a) // BLOCK for a, b in zip(at, at[1:])], device="cuda")
        s["block_decay"] = torch.repeat_interleave(torch.tensor(s["decay"], device="cuda"), blocks)[:, None]
        s["views"] = {k: [s[k][a:a + n] for a, n in zip(at, sizes)]
                      for k in ("param", "grad", "master", "m", "v") if s.get(k) is not None}
        for k in ("m_scale", "v_scale"):
            if k in s:
                s["views"][k] = [s[k][a // BLOCK:b // BLOCK] for a, b in zip(at, at[1:])]
    return s


def _rms(x):
    return torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)


def _plain(s):
    case = s["case"]
    op = case["op"]
    if op == "embed":
        return (s["E"][s["ids"].long()].float() * s["scale"]).to(TYPES[case["out"]])
    if op == "embed_grad":
        return s["dE"].index_add_(0, s["ids"], s["dout"].float() * s["scale"])
    if op == "norm":
        f = s["f"].float()
        y = f * _rms(f) * s["w_post"]
        if s["gate"] is not None:
            y = y * s["gate"][:, None]
        x = s["x"].float() * s["res_scale"] + y
        h = x * _rms(x) * s["w_pre"]
        return x.to(TYPES[case["x"]]), h.to(TYPES[case["h"]])
    if op == "norm_grad":
        x, f, dh = s["x"].float(), s["f"].float(), s["dh"]
        rx, rf = _rms(x), _rms(f)
        xn, fn = x * rx, f * rf
        dxn = dh * s["w_pre"]
        G = s["dx_out"] + rx * (dxn - xn * (dxn * xn).mean(-1, keepdim=True))
        s["dw_pre"] += (dh * xn).sum(0)
        dgate = (G * fn * s["w_post"]).sum(-1) if s["gate"] is not None else None
        dy = G if s["gate"] is None else G * s["gate"][:, None]
        s["dw_post"] += (dy * fn).sum(0)
        dfn = dy * s["w_post"]
        df = rf * (dfn - fn * (dfn * fn).mean(-1, keepdim=True))
        return {"dx": G * s["res_scale"], "df": df, "dgate": dgate, "dw_pre": s["dw_pre"], "dw_post": s["dw_post"]}
    b1, b2 = ADAM["beta1"], ADAM["beta2"]
    correct1, correct2 = 1 - b1 ** ADAM["step"], 1 - b2 ** ADAM["step"]
    g = s["grad"].float()
    if case["state"] == 32:
        m, v = s["m"], s["v"]
    else:
        m = (s["m"].float().view(-1, BLOCK) * s["m_scale"][:, None]).view(-1)
        v = (s["v"].float().view(-1, BLOCK) * s["v_scale"][:, None]).view(-1).square()
    m = m * b1 + g * (1 - b1)
    v = v * b2 + (g * g) * (1 - b2)
    root = v.sqrt()
    p = (s["master"] if s["master"] is not None else s["param"]).float().view(-1, BLOCK)
    step = (m / (root * (1 / math.sqrt(correct2)) + ADAM["eps"])).view(-1, BLOCK)
    p = (p - p * (s["block_decay"] * ADAM["lr"]) - step * (ADAM["lr"] / correct1)).view(-1)
    s["param"].copy_(p)
    if s["master"] is not None:
        s["master"].copy_(p)
    if case["state"] == 32:
        s["m"].copy_(m)
        s["v"].copy_(v)
    else:
        mb, rb = m.view(-1, BLOCK), root.view(-1, BLOCK)
        s["m_scale"].copy_((mb.abs().amax(1) * (1.0 / E4M3_MAX)).clamp_min(2.0 ** -120))
        s["v_scale"].copy_((rb.amax(1) * (1.0 / E4M3_MAX)).clamp_min(2.0 ** -120))
        s["m"].copy_((mb * s["m_scale"].reciprocal()[:, None]).view(-1))
        code = rb * s["v_scale"].reciprocal()[:, None]
        # a second moment that is not zero does not become zero
        s["v"].copy_(torch.where(rb > 0, code.clamp_min(2.0 ** -9), code).view(-1))
    return _adam_outputs(s)


def _adam_outputs(s):
    return {k: s[k] for k in ("param", "master", "m", "v", "m_scale", "v_scale") if s.get(k) is not None}


def _own(s):
    from mixture_lookup_experts_b200 import mole
    case = s["case"]
    op = case["op"]
    if op == "embed":
        return mole.mole_embed_forward(s["ids"], s["E"], s["scale"], out_dtype=TYPES[case["out"]])
    if op == "embed_grad":
        return mole.mole_embed_backward(s["ids"], s["dout"], s["dE"], s["scale"])
    if op == "norm":
        return mole.mole_block_norm_forward(s["x"], s["f"], w_post=s["w_post"], gate=s["gate"],
                                            res_scale=s["res_scale"], w_pre=s["w_pre"], eps=EPS,
                                            h_dtype=TYPES[case["h"]])
    if op == "norm_grad":
        dx, df, dgate = mole.mole_block_norm_backward(s["x"], s["dx_out"], s["dh"], s["f"], w_post=s["w_post"],
                                                      gate=s["gate"], res_scale=s["res_scale"], w_pre=s["w_pre"],
                                                      eps=EPS, dw_pre=s["dw_pre"], dw_post=s["dw_post"])
        return {"dx": dx, "df": df, "dgate": dgate, "dw_pre": s["dw_pre"], "dw_post": s["dw_post"]}
    v = s["views"]
    mole.mole_adamw_step(v["param"], v["grad"], v["m"], v["v"], masters=v.get("master"), m_scales=v.get("m_scale"),
                         v_scales=v.get("v_scale"), weight_decay=s["decay"], **ADAM)
    return _adam_outputs(s)


def run(state):
    return _own(state) if own else _plain(state)


def exact(case, seed):
    s = prepare(case, seed)
    d = {k: v.double() for k, v in s.items() if isinstance(v, torch.Tensor) and v.is_floating_point()
         and v.dtype != torch.float8_e4m3fn}
    op = case["op"]
    if op == "embed":
        return d["E"].index_select(0, s["ids"]) * s["scale"]
    if op == "embed_grad":
        order = torch.argsort(s["ids"], stable=True)
        rows, counts = torch.unique_consecutive(s["ids"][order], return_counts=True)
        total = torch.segment_reduce(d["dout"][order], "sum", lengths=counts, axis=0)
        d["dE"][rows.long()] += total * s["scale"]
        return d["dE"]
    if op in ("norm", "norm_grad"):
        x, f, gate = d["x"], d["f"], s["gate"]
        g = torch.ones(case["T"], 1, dtype=torch.float64, device="cuda") if gate is None else d["gate"][:, None]
        nf = (f.square().sum(1, keepdim=True) / case["D"] + EPS).sqrt()
        if op == "norm":
            x = s["res_scale"] * x + g * d["w_post"] * f / nf
            return x, d["w_pre"] * x / (x.square().sum(1, keepdim=True) / case["D"] + EPS).sqrt()
        # reverse mode on the definition
        leaf = {k: v.detach().requires_grad_() for k, v in
                {"x": x, "f": f, "g": g, "w_pre": d["w_pre"], "w_post": d["w_post"]}.items()}
        h = leaf["w_pre"] * leaf["x"] / (leaf["x"].square().sum(1, keepdim=True) / case["D"] + EPS).sqrt()
        Gx, Gw = torch.autograd.grad((h * d["dh"]).sum(), (leaf["x"], leaf["w_pre"]))
        G = Gx + d["dx_out"]
        y = leaf["g"] * leaf["w_post"] * leaf["f"] / (leaf["f"].square().sum(1, keepdim=True) / case["D"] + EPS).sqrt()
        Gf, Gg, Gp = torch.autograd.grad((y * G).sum(), (leaf["f"], leaf["g"], leaf["w_post"]))
        return {"dx": s["res_scale"] * G, "df": Gf, "dgate": None if gate is None else Gg[:, 0],
                "dw_pre": d["dw_pre"] + Gw, "dw_post": d["dw_post"] + Gp}
    b1, b2, t = ADAM["beta1"], ADAM["beta2"], ADAM["step"]
    spread = lambda scale: scale.double().repeat_interleave(BLOCK)  # noqa: E731
    if case["state"] == 32:
        m, v = d["m"], d["v"]
    else:
        m, v = s["m"].double() * spread(s["m_scale"]), (s["v"].double() * spread(s["v_scale"])) ** 2
    m, v = b1 * m + (1 - b1) * d["grad"], b2 * v + (1 - b2) * d["grad"] ** 2
    p = d["master"] if s["master"] is not None else d["param"]
    p = (p.view(-1, BLOCK) * (1 - ADAM["lr"] * s["block_decay"].double())).view(-1)
    p = p - ADAM["lr"] * (m / (1 - b1 ** t)) / ((v / (1 - b2 ** t)).sqrt() + ADAM["eps"])
    out = {"param": p}
    if s["master"] is not None:
        out["master"] = p
    if case["state"] == 32:
        out["m"], out["v"] = m, v
    else:
        for name, w in (("m", m), ("v", v.sqrt())):
            scale = w.view(-1, BLOCK).abs().amax(1) / E4M3_MAX
            out[name] = w / spread(scale.clamp_min(1e-300))
            out[name + "_scale"] = scale.clamp_min(2.0 ** -120)
    return out

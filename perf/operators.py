"""The operators of a pre-norm MLP branch over a packed token buffer: the
modality-specific layer norm, the linear layer with bias, activation and residual
in its epilogue, their backward passes, and activation checkpoints in 8 bits.

A pack is ``samples``: "frames,grid_h,grid_w,n_text" per sample, joined by ";".
Every sample's image tokens come first, then its text tokens; image tokens use
parameter set 0, text tokens set 1.
"""

import math

import torch

own = False

HID = 24 * 128      # width of the full-size packs: 24 heads x 128
WIDE = 4 * HID      # their MLP width
BLOCK = 128         # channels per scale of an 8-bit checkpoint
EPS = 1e-6
ACTS = {"none": 0, "gelu": 1, "silu": 2}

TINY_PACK = "1,16,16,20;1,8,32,12"                                             # 544 tokens
TRAIN_PACK = "1,64,64,160;1,32,128,160;1,48,48,160;1,32,32,160;0,0,0,4224"     # 16384 tokens, padded
CFG_PACK = "1,64,64,256;1,64,64,16"                                            # 8464 tokens


def listed():
    return [
        # the embedding norm of one short prompt: a launch and little else
        dict(name="ln_prompt", op="ln", samples="0,0,0,20", hid=128),
        # the pre-MLP norm of a full training pack
        dict(name="ln_train", op="ln", samples=TRAIN_PACK, hid=HID),
        # its backward, the residual path's gradient added, from the kept bf16 input
        dict(name="ln_bwd_train", op="ln_bwd", samples=TRAIN_PACK, hid=HID, ckpt=False, resid=True),
        # an odd pack and width, the input kept in 8 bits
        dict(name="ln_bwd_odd_ckpt", op="ln_bwd", samples="1,37,61,77;1,29,53,1;0,0,0,313;1,1,643,9",
             hid=1000, ckpt=True, resid=False),
        # text conditioning at inference: one prompt through an MLP's first layer
        dict(name="linear_prompt", op="linear", samples="0,0,0,16", K=HID, N=WIDE, act="gelu",
             bias=True, resid=False, keep="no"),
        # MLP up projection of the two guidance branches, pre-activations kept in 8 bits
        dict(name="linear_cfg_up", op="linear", samples=CFG_PACK, K=HID, N=WIDE, act="gelu",
             bias=True, resid=False, keep="8bit"),
        # an adapter's output projection: odd pack and widths, residual, z kept in bf16
        dict(name="linear_odd_resid", op="linear", samples="1,31,33,7;1,17,91,45;0,0,0,129", K=1000,
             N=2056, act="silu", bias=True, resid=True, keep="bf16"),
        # MLP down projection backward of the guidance pack, its input kept in 8 bits
        dict(name="linear_bwd_cfg_down", op="linear_bwd", samples=CFG_PACK, K=WIDE, N=HID,
             act="none", xkeep="8bit", zkeep="no"),
        # adapter backward at odd sizes, everything kept in bf16
        dict(name="linear_bwd_odd", op="linear_bwd", samples="1,31,33,7;1,17,91,45;0,0,0,129",
             K=1000, N=2056, act="silu", xkeep="bf16", zkeep="bf16"),
        # the first layer of a small model's MLP: few rows, everything kept in 8 bits
        dict(name="linear_bwd_tiny", op="linear_bwd", samples=TINY_PACK, K=128, N=512, act="gelu",
             xkeep="8bit", zkeep="8bit"),
        # a small model's checkpoint, stored and read back
        dict(name="ckpt_tiny", op="ckpt", samples=TINY_PACK, C=512, act="none"),
        # the MLP pre-activations of a training pack, read back through the GELU
        dict(name="ckpt_train", op="ckpt", samples=TRAIN_PACK, C=WIDE, act="gelu"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _draw_pack(rng, most):
    """A pack of at most ``most`` tokens whose size is spread over its logarithm."""
    left = _log_int(rng, 1, most)
    rows = []
    for _ in range(rng.randint(1, 5)):
        if left < 1:
            break
        n = rng.randint(1, left)
        text = min(n, rng.choice((0, 1, n, _log_int(rng, 1, n))))
        h = _log_int(rng, 1, max(1, n - text))
        w = (n - text) // h
        rows.append("%d,%d,%d,%d" % ((1, h, w, text) if w else (0, 0, 0, text)))
        left -= h * w + text
    return ";".join(rows)


def draw(rng):
    op = rng.choice(("ln", "ln_bwd", "linear", "linear", "linear_bwd", "linear_bwd", "ckpt"))
    if op in ("ln", "ln_bwd"):
        case = dict(op=op, samples=_draw_pack(rng, 16384), hid=8 * _log_int(rng, 2, HID // 8))
        if op == "ln_bwd":
            case.update(ckpt=rng.random() < 0.5, resid=rng.random() < 0.5)
        return case
    if op == "ckpt":
        return dict(op=op, samples=_draw_pack(rng, 8464), C=8 * _log_int(rng, 1, WIDE // 8),
                    act=rng.choice(tuple(ACTS)))
    # widths in eights, one of them at most the full MLP width
    a, b = 8 * _log_int(rng, 4, WIDE // 8), 8 * _log_int(rng, 4, HID // 8)
    K, N = (a, b) if rng.random() < 0.5 else (b, a)
    case = dict(op=op, samples=_draw_pack(rng, 8464), K=K, N=N, act=rng.choice(tuple(ACTS)))
    if op == "linear":
        case.update(bias=rng.random() < 0.7, resid=rng.random() < 0.5,
                    keep=rng.choice(("no", "bf16", "8bit")))
    else:
        case.update(xkeep=rng.choice(("bf16", "8bit")),
                    zkeep="no" if case["act"] == "none" else rng.choice(("bf16", "8bit")))
    return case


def _samples(case):
    return [tuple(int(v) for v in s.split(",")) for s in case["samples"].split(";")]


def _counts(case):
    img = sum(f * h * w for f, h, w, _ in _samples(case))
    return img, sum(t for _, _, _, t in _samples(case))


def work(case):
    img, txt = _counts(case)
    T, sets = img + txt, (img > 0) + (txt > 0)
    op = case["op"]
    if op == "ln":
        h = case["hid"]
        return {"bytes": 4 * T * h + 8 * sets * h + 9 * T, "flops": 8 * T * h}
    if op == "ln_bwd":
        h = case["hid"]
        x = (1 + 4 / BLOCK) if case["ckpt"] else 2
        return {"bytes": T * h * (4 + x + (2 if case["resid"] else 0)) + 4 * sets * h + 16 * h + 9 * T,
                "flops": 16 * T * h}
    if op == "ckpt":
        return {"bytes": T * case["C"] * (6 + 8 / BLOCK), "flops": 6 * T * case["C"]}
    K, N = case["K"], case["N"]
    kept = {"no": 0, "bf16": 2, "8bit": 1 + 4 / BLOCK}
    if op == "linear":
        return {"bytes": 2 * T * K + 2 * sets * K * N + T * N * (2 + kept[case["keep"]]
                                                                  + (2 if case["resid"] else 0)),
                "flops": 2 * T * K * N}
    return {"bytes": T * K * (2 + kept[case["xkeep"]]) + T * N * (2 + kept[case["zkeep"]])
            + 2 * sets * K * N + 4 * K * N + 8 * N, "flops": 4 * T * K * N}


# ------------------------------------------------------------------ inputs
def _normal(gen, shape, scale=1.0, dtype=torch.bfloat16):
    x = torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32)
    return (x * scale).to(dtype)


def _store8(x):
    """An 8-bit checkpoint of x [T][C] in fp32: codes and one scale per 128 channels."""
    T, C = x.shape
    nb = -(-C // BLOCK)
    b = torch.nn.functional.pad(x.float(), (0, nb * BLOCK - C)).view(T, nb, BLOCK)
    amax = b.abs().amax(-1)
    zero, bad = amax < 2.0 ** -100, ~torch.isfinite(amax)
    inv = torch.where(zero | bad, torch.zeros_like(amax), 127.0 / amax)
    s = torch.where(zero, torch.zeros_like(amax), amax / 127.0)
    s = torch.where(bad, torch.full_like(s, float("nan")), s)
    q = torch.where(bad[..., None], torch.zeros_like(b), torch.round(b * inv[..., None]))
    return q.clamp(-127, 127).to(torch.int8).view(T, nb * BLOCK)[:, :C].contiguous(), s


def _load8(q, s):
    T, C = q.shape
    return q.float() * s.repeat_interleave(BLOCK, 1)[:, :C]


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    mods = []
    for f, h, w, t in _samples(case):
        mods += [0] * (f * h * w) + [1] * t
    tok_mod = torch.tensor(mods, dtype=torch.uint8)
    T = len(mods)
    st = dict(case=dict(case), T=T, samples=_samples(case), tok_mod=tok_mod.cuda(),
              img=torch.nonzero(tok_mod == 0).flatten().cuda(),
              txt=torch.nonzero(tok_mod == 1).flatten().cuda(), hold={})
    op = case["op"]
    if op in ("ln", "ln_bwd"):
        hid = case["hid"]
        # residual-stream rows: unit spread around a small offset of their own
        st["x"] = (_normal(gen, (T, hid), dtype=torch.float32)
                   + _normal(gen, (T, 1), 0.3, torch.float32)).to(torch.bfloat16)
        st["gamma"] = 1 + _normal(gen, (2, hid), 0.1, torch.float32)
        st["beta"] = _normal(gen, (2, hid), 0.1, torch.float32)
        if op == "ln_bwd":
            st["dy"] = _normal(gen, (T, hid))
            st["resid"] = _normal(gen, (T, hid)) if case["resid"] else None
            st["x8"], st["xs"] = _store8(st["x"]) if case["ckpt"] else (None, None)
            x = (_load8(st["x8"], st["xs"]) if case["ckpt"] else st["x"]).double()
            var, mean = torch.var_mean(x, 1, correction=0)
            st["stats"] = torch.stack((mean, (var + EPS).rsqrt()), 1).float()
            if case["ckpt"]:
                st["x"] = None
    elif op == "ckpt":
        st["x"] = _normal(gen, (T, case["C"]))
    else:
        K, N = case["K"], case["N"]
        st["W"] = _normal(gen, (2, N, K), 1 / math.sqrt(K))
        if op == "linear":
            st["x"] = _normal(gen, (T, K))
            st["bias"] = _normal(gen, (2, N), 0.1, torch.float32) if case["bias"] else None
            st["resid"] = _normal(gen, (T, N)) if case["resid"] else None
        else:
            x, z = _normal(gen, (T, K)), _normal(gen, (T, N))
            st["dout"] = _normal(gen, (T, N))
            st["x"], st["x8"], st["xs"] = (x, None, None) if case["xkeep"] == "bf16" else (None, *_store8(x))
            st["z"], st["z8"], st["zs"] = {"no": lambda: (None, None, None), "bf16": lambda: (z, None, None),
                                           "8bit": lambda: (None, *_store8(z))}[case["zkeep"]]()
    return st


# ------------------------------------------------------------- plain forms
def _act(z, act):
    if act == "gelu":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z)))
    return z / (1 + torch.exp(-z)) if act == "silu" else z


def _act_grad(z, act):
    if act == "gelu":
        th = torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z))
        return 0.5 * (1 + th) + 0.5 * z * (1 - th * th) * math.sqrt(2 / math.pi) * (1 + 3 * 0.044715 * z * z)
    s = 1 / (1 + torch.exp(-z))
    return s * (1 + z * (1 - s))


def _plain_ln(st):
    x, m = st["x"].float(), st["tok_mod"].long()
    mean = x.mean(1, keepdim=True)
    xc = x - mean
    rstd = 1 / torch.sqrt((xc * xc).mean(1, keepdim=True) + EPS)
    y = xc * rstd * st["gamma"][m] + st["beta"][m]
    return {"y": y.to(torch.bfloat16), "stats": torch.cat((mean, rstd), 1)}


def _plain_ln_bwd(st):
    x = st["x"].float() if st["x"] is not None else _load8(st["x8"], st["xs"])
    dy, rstd = st["dy"].float(), st["stats"][:, 1:]
    xh = (x - st["stats"][:, :1]) * rstd
    g = dy * st["gamma"][st["tok_mod"].long()]
    dx = (g - g.mean(1, keepdim=True) - xh * (g * xh).mean(1, keepdim=True)) * rstd
    if st["resid"] is not None:
        dx = dx + st["resid"].float()
    p = dy * xh
    return {"dx": dx.to(torch.bfloat16),
            "dgamma": torch.stack((p[st["img"]].sum(0), p[st["txt"]].sum(0))),
            "dbeta": torch.stack((dy[st["img"]].sum(0), dy[st["txt"]].sum(0)))}


def _plain_linear(st):
    c, x, W = st["case"], st["x"].float(), st["W"].float()
    z = torch.empty((st["T"], c["N"]), device="cuda")
    z[st["img"]] = x[st["img"]] @ W[0].T
    z[st["txt"]] = x[st["txt"]] @ W[1].T
    if st["bias"] is not None:
        z = z + st["bias"][st["tok_mod"].long()]
    out = _act(z, c["act"])
    if st["resid"] is not None:
        out = out + st["resid"].float()
    kept = z if c["keep"] == "bf16" else _load8(*_store8(z)) if c["keep"] == "8bit" else None
    return {"out": out.to(torch.bfloat16), "z": None if kept is None else kept.to(torch.bfloat16)}


def _plain_linear_bwd(st):
    c, W, i, t = st["case"], st["W"].float(), st["img"], st["txt"]
    x = st["x"].float() if st["x"] is not None else _load8(st["x8"], st["xs"])
    dz = st["dout"].float()
    if c["act"] != "none":
        dz = dz * _act_grad(st["z"].float() if st["z"] is not None else _load8(st["z8"], st["zs"]), c["act"])
    dx = torch.empty((st["T"], c["K"]), device="cuda")
    dx[i] = dz[i] @ W[0]
    dx[t] = dz[t] @ W[1]
    return {"dx": dx.to(torch.bfloat16),
            "dW": torch.stack((dz[i].T @ x[i], dz[t].T @ x[t])).to(torch.bfloat16),
            "db": torch.stack((dz[i].sum(0), dz[t].sum(0)))}


def _plain_ckpt(st):
    q, s = _store8(st["x"])
    return {"y": _act(_load8(q, s), st["case"]["act"]).to(torch.bfloat16), "scale": s}


# ------------------------------------------------- the framework's operators
def _held(st, name, shape, dtype=torch.bfloat16):
    """A buffer that the caller owns: made on the first pass, used again after."""
    if name not in st["hold"]:
        st["hold"][name] = torch.empty(shape, dtype=dtype, device="cuda")
    return st["hold"][name]


def _plan(st, mf):
    if "descs" not in st["hold"]:
        st["hold"]["descs"] = mf.make_descs(st["samples"])
    return st["hold"]["descs"]


def _own_ln(st, mf):
    T, hid = st["T"], st["case"]["hid"]
    y, stats = _held(st, "y", (T, hid)), _held(st, "stats", (T, 2), torch.float32)
    mf.mf_layer_norm(st["x"], st["gamma"], st["beta"], st["tok_mod"], T, hid, EPS, y, stats)
    return {"y": y, "stats": stats}


def _own_ln_bwd(st, mf):
    T, hid = st["T"], st["case"]["hid"]
    dx = _held(st, "dx", (T, hid))
    dgamma, dbeta = (_held(st, n, (2, hid), torch.float32) for n in ("dgamma", "dbeta"))
    nws = mf.mf_layer_norm_bwd_workspace_size(T, hid)
    mf.mf_layer_norm_bwd(st["dy"], st["x"], st["x8"], st["xs"], st["gamma"], st["stats"],
                         st["tok_mod"], st["resid"], T, hid, dx, dgamma, dbeta,
                         _held(st, "ws", (nws,), torch.uint8), nws)
    return {"dx": dx, "dgamma": dgamma, "dbeta": dbeta}


def _own_linear(st, mf):
    c, T = st["case"], st["T"]
    K, N = c["K"], c["N"]
    out = _held(st, "out", (T, N))
    z = _held(st, "z", (T, N)) if c["keep"] != "no" else None
    z8 = _held(st, "z8", (T, N), torch.int8) if c["keep"] == "8bit" else None
    zs = _held(st, "zs", (T, -(-N // BLOCK)), torch.float32) if c["keep"] == "8bit" else None
    mf.mf_linear_fused(st["x"], st["W"], st["bias"], st["resid"], st["tok_mod"], _plan(st, mf), K, N,
                       ACTS[c["act"]], z if c["keep"] == "bf16" else None, z8, zs, out)
    if c["keep"] == "8bit":
        mf.mf_act8_dequantize(z8, zs, T, N, mf.MF_ACT_NONE, z)
    return {"out": out, "z": z}


def _own_linear_bwd(st, mf):
    c, T = st["case"], st["T"]
    K, N = c["K"], c["N"]
    dx, dW = _held(st, "dx", (T, K)), _held(st, "dW", (2, N, K))
    db = _held(st, "db", (2, N), torch.float32)
    nws = mf.mf_linear_fused_bwd_workspace_size(T, K, N)
    mf.mf_linear_fused_bwd(st["dout"], st["x"], st["x8"], st["xs"], st["W"], st["z"], st["z8"], st["zs"],
                           st["tok_mod"], _plan(st, mf), K, N, ACTS[c["act"]], dx, dW, db,
                           _held(st, "ws", (nws,), torch.uint8), nws)
    return {"dx": dx, "dW": dW, "db": db}


def _own_ckpt(st, mf):
    T, C = st["T"], st["case"]["C"]
    q, y = _held(st, "q", (T, C), torch.int8), _held(st, "y", (T, C))
    s = _held(st, "s", (T, -(-C // BLOCK)), torch.float32)
    mf.mf_act8_quantize(st["x"], T, C, q, s)
    mf.mf_act8_dequantize(q, s, T, C, ACTS[st["case"]["act"]], y)
    return {"y": y, "scale": s}


PLAIN = {"ln": _plain_ln, "ln_bwd": _plain_ln_bwd, "linear": _plain_linear,
         "linear_bwd": _plain_linear_bwd, "ckpt": _plain_ckpt}
OWN = {"ln": _own_ln, "ln_bwd": _own_ln_bwd, "linear": _own_linear,
       "linear_bwd": _own_linear_bwd, "ckpt": _own_ckpt}


def run(state):
    if own:
        import resolution_packed_diffusion_b200 as mf
        return OWN[state["case"]["op"]](state, mf)
    return PLAIN[state["case"]["op"]](state)


# ------------------------------------------------------- 64-bit definitions
def _exact_codes(x):
    """Values of the 8-bit checkpoint of x, from its definition."""
    out = torch.empty_like(x)
    for c in range(0, x.shape[1], BLOCK):
        blk = x[:, c:c + BLOCK]
        top = blk.abs().max(1, keepdim=True).values
        step = top / 127
        out[:, c:c + BLOCK] = torch.where(top < 2.0 ** -100, torch.zeros_like(blk),
                                          torch.round(blk / step.clamp_min(2.0 ** -120)) * step)
    return out


def _exact_value(codes, scale):
    C = codes.shape[1]
    return codes.double() * scale.double()[:, torch.arange(C, device="cuda") // BLOCK]


def _exact_act(z, act):
    """(act(z), act'(z)): GELU's tanh form as z sigma(2u), SiLU as z sigma(z)."""
    if act == "none":
        return z, torch.ones_like(z)
    c = 2 * math.sqrt(2 / math.pi) if act == "gelu" else 1.0
    a = 0.044715 if act == "gelu" else 0.0
    s = torch.sigmoid(c * (z + a * z ** 3))
    return z * s, s + z * s * (1 - s) * c * (1 + 3 * a * z * z)


def exact(case, seed):
    st = prepare(case, seed)
    op, sel = case["op"], [st["tok_mod"] == m for m in (0, 1)]
    if op == "ckpt":
        x = st["x"].double()
        tops = [x[:, c:c + BLOCK].abs().max(1).values for c in range(0, x.shape[1], BLOCK)]
        return {"y": _exact_act(_exact_codes(x), case["act"])[0], "scale": torch.stack(tops, 1) / 127}
    if op == "ln":
        x = st["x"].double()
        y, stats = torch.empty_like(x), torch.empty((st["T"], 2), dtype=torch.float64, device="cuda")
        stats[:, 0] = x.sum(1) / x.shape[1]
        dev = x - stats[:, :1]
        stats[:, 1] = (dev.square().sum(1) / x.shape[1] + EPS) ** -0.5
        for m in (0, 1):
            y[sel[m]] = (dev * stats[:, 1:])[sel[m]] * st["gamma"][m].double() + st["beta"][m].double()
        return {"y": y, "stats": stats}
    if op == "ln_bwd":
        x = st["x"].double() if st["x"] is not None else _exact_value(st["x8"], st["xs"])
        dy, n = st["dy"].double(), x.shape[1]
        mu, r = st["stats"].double().split(1, 1)
        xh = (x - mu) * r
        dx, dgamma, dbeta = torch.empty_like(x), [], []
        for m in (0, 1):
            d, h = dy[sel[m]], xh[sel[m]]
            dgamma.append(torch.einsum("tc,tc->c", d, h))
            dbeta.append(d.sum(0))
            g = d * st["gamma"][m].double()
            dots = torch.einsum("tc,tc->t", g, h)
            dx[sel[m]] = r[sel[m]] * (g - g.sum(1, keepdim=True) / n - h * dots[:, None] / n)
        if st["resid"] is not None:
            dx += st["resid"].double()
        return {"dx": dx, "dgamma": torch.stack(dgamma), "dbeta": torch.stack(dbeta)}
    W = st["W"].double()
    if op == "linear":
        x = st["x"].double()
        z = torch.empty((st["T"], case["N"]), dtype=torch.float64, device="cuda")
        for m in (0, 1):
            z[sel[m]] = torch.einsum("tk,nk->tn", x[sel[m]], W[m])
            if st["bias"] is not None:
                z[sel[m]] += st["bias"][m].double()
        out = _exact_act(z, case["act"])[0]
        if st["resid"] is not None:
            out = out + st["resid"].double()
        return {"out": out, "z": {"no": lambda v: None, "bf16": lambda v: v, "8bit": _exact_codes}[case["keep"]](z)}
    x = st["x"].double() if st["x"] is not None else _exact_value(st["x8"], st["xs"])
    dz = st["dout"].double()
    if case["act"] != "none":
        z = st["z"].double() if st["z"] is not None else _exact_value(st["z8"], st["zs"])
        dz = dz * _exact_act(z, case["act"])[1]
    dx, dW, db = torch.empty_like(x), [], []
    for m in (0, 1):
        dx[sel[m]] = torch.einsum("tn,nk->tk", dz[sel[m]], W[m])
        dW.append(torch.einsum("tn,tk->nk", dz[sel[m]], x[sel[m]]))
        db.append(dz[sel[m]].sum(0))
    return {"dx": dx, "dW": torch.stack(dW), "db": torch.stack(db)}

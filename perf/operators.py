"""The block operators around and beside the gated FFN, as a benchmark calls them.

Three families: the norms before and after a block with its gate and residual
(norm_fwd, norm_bwd), activation checkpoints in 8 bits (ckpt8: written and read
back; act8: the activation's backward from them) and the mixture-of-experts
layer for a few tokens (moe).  `own` selects the library's calls; otherwise the
same operators in elementary torch operations in FP32, rounded once at the end.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
BLOCK = 64  # columns that share one 8-bit scale
EPS = 1e-6


def listed():
    return [
        # decode of one token through a layer: the norm pair between two blocks, latency only
        {"name": "norm_fwd_1x4096", "op": "norm_fwd", "M": 1, "H": 4096, "dtype": "bf16", "gate": "none", "alpha": 1.0},
        # the training step's 4096 tokens (8 sequences of 512), sandwich norms with a per-channel gate
        {"name": "norm_fwd_4096x4096", "op": "norm_fwd", "M": 4096, "H": 4096, "dtype": "bf16", "gate": "row", "alpha": 1.0},
        # the same step's backward, weight and gate gradients among the outputs
        {"name": "norm_bwd_4096x4096", "op": "norm_bwd", "M": 4096, "H": 4096, "dtype": "bf16", "gate": "row", "alpha": 1.0},
        # odd width and token count, a gate for every token and channel (conditioned blocks), scaled residual, FP16
        {"name": "norm_bwd_1003x5125", "op": "norm_bwd", "M": 1003, "H": 5125, "dtype": "fp16", "gate": "full", "alpha": 0.7071},
        # a small batch's saved activation, written and read back: latency
        {"name": "ckpt8_32x12288", "op": "ckpt8", "M": 32, "N": 12288, "dtype": "bf16"},
        # what the training step saves of one projection, written and read back
        {"name": "ckpt8_4096x12288", "op": "ckpt8", "M": 4096, "N": 12288, "dtype": "bf16"},
        # the activation's backward in the training step, from both saved projections
        {"name": "act8_4096x12288", "op": "act8", "M": 4096, "N": 12288, "dtype": "bf16"},
        # ragged: the last block of each row is short, FP16
        {"name": "act8_777x5461", "op": "act8", "M": 777, "N": 5461, "dtype": "fp16"},
        # serving one token: eight of many small experts
        {"name": "moe_1_e128k8", "op": "moe", "M": 1, "H": 2048, "I": 768, "E": 128, "k": 8, "renorm": True, "dtype": "bf16"},
        # a serving batch of 32 over the same experts: nearly every expert is read
        {"name": "moe_32_e128k8", "op": "moe", "M": 32, "H": 2048, "I": 768, "E": 128, "k": 8, "renorm": True, "dtype": "bf16"},
        # a batch of 8 over a few experts of the dense FFN's own size
        {"name": "moe_8_e8k2", "op": "moe", "M": 8, "H": 4096, "I": 12288, "E": 8, "k": 2, "renorm": True, "dtype": "bf16"},
        # odd sizes, weights of the whole softmax, FP16
        {"name": "moe_5_e60k4", "op": "moe", "M": 5, "H": 1003, "I": 1411, "E": 60, "k": 4, "renorm": False, "dtype": "fp16"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm_fwd", "norm_bwd", "ckpt8", "act8", "moe", "moe"])
    dtype = rng.choice(["bf16", "fp16"])
    if op in ("norm_fwd", "norm_bwd"):
        H = _log(rng, 64, 16384)
        M = _log(rng, 1, min(16384, (1 << 24) // H))
        return {"op": op, "M": M, "H": H, "dtype": dtype, "gate": rng.choice(["none", "row", "full"]),
                "alpha": rng.choice([1.0, 0.5])}
    if op in ("ckpt8", "act8"):
        N = _log(rng, 64, 28672)
        return {"op": op, "M": _log(rng, 1, min(8192, (1 << 25) // N)), "N": N, "dtype": dtype}
    k = rng.choice([1, 2, 4, 8])
    E = max(2 * k, _log(rng, 4, 256))
    H = _log(rng, 256, 8192)
    I = _log(rng, 128, max(129, min(12288, (1 << 28) // (E * H))))
    M = _log(rng, 1, min(64, max(1, (1 << 29) // (k * H * I))))
    return {"op": op, "M": M, "H": H, "I": I, "E": E, "k": k, "renorm": rng.random() < 0.5,
            "dtype": dtype}


def _rows(gen, shape, dtype, scale=1.0, shift=0.0):
    """Normal values, row-major with a leading dimension that is a multiple of 8 elements."""
    *lead, cols = shape
    buf = torch.empty((*lead, -(-cols // 8) * 8), dtype=dtype, device="cuda")
    buf.normal_(shift, scale, generator=gen)
    return buf[..., :cols]


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dt = DTYPES[case["dtype"]]
    st = {"case": case, "dtype": dt}
    if case["op"] in ("norm_fwd", "norm_bwd"):
        M, H = case["M"], case["H"]
        st["res"] = _rows(gen, (M, H), dt, 1.5)
        st["y"] = _rows(gen, (M, H), dt, 0.5)
        st["w_post"] = _rows(gen, (H,), dt, 0.1, 1.0)
        st["w_next"] = _rows(gen, (H,), dt, 0.1, 1.0)
        st["gate"] = {"none": lambda: None, "row": lambda: _rows(gen, (H,), dt, 0.3, 0.5),
                      "full": lambda: _rows(gen, (M, H), dt, 0.3, 0.5)}[case["gate"]]()
        if case["op"] == "norm_bwd":  # what the forward left: the new residual and the two scales of each row
            yf, gate = st["y"].float(), 1.0 if st["gate"] is None else st["gate"].float()
            r_y = torch.rsqrt((yf * yf).mean(1) + EPS)
            z = case["alpha"] * st["res"].float() + gate * (yf * r_y[:, None] * st["w_post"].float())
            r_z = torch.rsqrt((z * z).mean(1) + EPS)
            st["z"] = _rows(gen, (M, H), dt)
            st["z"].copy_(z)
            st["rstd"] = torch.stack((r_y, r_z), 1).contiguous()
            st["dz"] = _rows(gen, (M, H), dt, 0.1)
            st["dh"] = _rows(gen, (M, H), dt, 0.1)
    elif case["op"] in ("ckpt8", "act8"):
        M, N = case["M"], case["N"]
        st["g"] = _rows(gen, (M, N), dt, 1.3)
        if case["op"] == "act8":  # the codes and scales that the forward kept
            st["u"] = _rows(gen, (M, N), dt, 1.3)
            st["da"] = _rows(gen, (M, N), dt, 0.1)
            st["g8"], st["u8"] = _quantise(st["g"]), _quantise(st["u"])
    else:
        M, H, I, E = (case[n] for n in ("M", "H", "I", "E"))
        st["x"] = _rows(gen, (M, H), dt)
        st["w_router"] = _rows(gen, (E, H), dt, 1.0 / math.sqrt(H))
        st["w_gate"] = _rows(gen, (E, I, H), dt, 1.0 / math.sqrt(H))
        st["w_up"] = _rows(gen, (E, I, H), dt, 1.0 / math.sqrt(H))
        st["w_down"] = _rows(gen, (E, H, I), dt, 1.0 / math.sqrt(I))
    return st


def _blocks(t):
    """[M, N] -> [M, blocks, BLOCK] in FP32, the last block padded with zeros."""
    M, N = t.shape
    nb = -(-N // BLOCK)
    return torch.nn.functional.pad(t.float(), (0, nb * BLOCK - N)).view(M, nb, BLOCK)


def _quantise(t):
    """(codes [M, N] int8, scales [M, blocks] FP32): scale = largest magnitude / 127, code = value * (127 / largest) to nearest even."""
    M, N = t.shape
    b = _blocks(t)
    top = b.abs().amax(2)
    s = top / 127.0
    q = torch.round(b * torch.where(top > 0, 127.0 / top, 0.0)[..., None])
    ld = -(-N // 16) * 16
    codes = torch.zeros((M, ld), dtype=torch.int8, device=t.device)[:, :N]
    codes.copy_(q.clamp(-127, 127).view(M, -1)[:, :N])
    return codes, s


def _read_back(codes, s):
    M, N = codes.shape
    return (_blocks(codes) * s[..., None]).view(M, -1)[:, :N]


def run(st):
    return (_own if own else _plain)(st)


def _own(st):
    from deterministic_gated_ffn_amd import binding as dgf
    case = st["case"]
    if case["op"] == "norm_fwd":
        r = dgf.norm_fwd(st["res"], st["y"], w_post=st["w_post"], gate=st["gate"], alpha=case["alpha"],
                         w_next=st["w_next"], eps=EPS, training=True)
        return {"z": r["z"], "h": r["h"], "rstd": r["rstd"]}
    if case["op"] == "norm_bwd":
        return dgf.norm_bwd(st["dz"], st["dh"], st["z"], st["y"], w_post=st["w_post"], gate=st["gate"],
                            alpha=case["alpha"], w_next=st["w_next"], rstd=st["rstd"])
    if case["op"] == "ckpt8":
        return dgf.unpack8(dgf.pack8(st["g"]))
    if case["op"] == "act8":
        dg, du, a = dgf.act_bwd_q8(st["da"], dgf.Packed8(*st["g8"], st["dtype"]), dgf.Packed8(*st["u8"], st["dtype"]))
        return {"dg": dg, "du": du, "a": a}
    y, _, p = dgf.moe_fwd(st["x"], st["w_router"], st["w_gate"], st["w_up"], st["w_down"], case["k"],
                          renorm=case["renorm"], routing=True)
    return {"y": y, "p": p}


def _plain(st):
    case, dt = st["case"], st["dtype"]
    if case["op"] == "norm_fwd":
        y, res = st["y"].float(), st["res"].float()
        r_y = torch.rsqrt((y * y).mean(1, keepdim=True) + EPS)
        t = y * r_y * st["w_post"].float()
        z = case["alpha"] * res + (t if st["gate"] is None else st["gate"].float() * t)
        r_z = torch.rsqrt((z * z).mean(1, keepdim=True) + EPS)
        return {"z": z.to(dt), "h": (z * r_z * st["w_next"].float()).to(dt), "rstd": torch.cat((r_y, r_z), 1)}
    if case["op"] == "norm_bwd":
        y, z, dh = st["y"].float(), st["z"].float(), st["dh"].float()
        r_y, r_z = st["rstd"][:, :1], st["rstd"][:, 1:]
        dn = dh * st["w_next"].float()
        G = st["dz"].float() + r_z * (dn - z * (r_z * r_z * (dn * z).mean(1, keepdim=True)))
        yn = y * r_y
        dgate = G * (yn * st["w_post"].float())
        dt_ = G if st["gate"] is None else G * st["gate"].float()
        dq = dt_ * st["w_post"].float()
        out = {"dres": (case["alpha"] * G).to(dt),
               "dy": (r_y * (dq - yn * (dq * yn).mean(1, keepdim=True))).to(dt),
               "dw_post": (dt_ * yn).sum(0).to(dt), "dw_next": (dh * z * r_z).sum(0).to(dt)}
        if st["gate"] is not None:
            out["dgate"] = (dgate.sum(0) if case["gate"] == "row" else dgate).to(dt)
        return out
    if case["op"] == "ckpt8":
        return _read_back(*_quantise(st["g"])).to(dt)
    if case["op"] == "act8":
        g, u, da = _read_back(*st["g8"]), _read_back(*st["u8"]), st["da"].float()
        s = 1.0 / (1.0 + torch.exp(-g))
        silu = g * s
        return {"dg": (da * u * (s * (1.0 + g * (1.0 - s)))).to(dt), "du": (da * silu).to(dt), "a": (silu * u).to(dt)}
    M, H, I, k = (case[n] for n in ("M", "H", "I", "k"))
    x = st["x"].float()
    logits = x @ st["w_router"].float().t()
    p, order = torch.sort(torch.softmax(logits, 1), dim=1, descending=True, stable=True)
    p, ids = p[:, :k], order[:, :k].reshape(-1)
    if case["renorm"]:
        p = p / p.sum(1, keepdim=True)
    xk = x.repeat_interleave(k, 0).unsqueeze(2)
    g = torch.bmm(st["w_gate"][ids].float(), xk)
    u = torch.bmm(st["w_up"][ids].float(), xk)
    a = g / (1.0 + torch.exp(-g)) * u
    o = torch.bmm(st["w_down"][ids].float(), a).view(M, k, H)
    return {"y": (o * p[:, :, None]).sum(1).to(dt), "p": p.contiguous()}


def work(case):
    """Bytes: each input read once, each output written once.  An expert's weights are
    read once however many tokens chose it: E (1 - (1 - k/E)^M) experts on average."""
    op, M = case["op"], case["M"]
    if op in ("norm_fwd", "norm_bwd"):
        H, full, row = case["H"], case["gate"] == "full", case["gate"] == "row"
        if op == "norm_fwd":
            return {"bytes": M * H * 2 * (4 + full) + H * 2 * (2 + row) + 8 * M, "flops": 12 * M * H}
        return {"bytes": M * H * 2 * (6 + 2 * full) + H * 2 * (4 + 2 * row) + 8 * M, "flops": 30 * M * H}
    if op in ("ckpt8", "act8"):
        N = case["N"]
        packed = M * N + 4 * M * -(-N // BLOCK)
        if op == "ckpt8":
            return {"bytes": 4 * M * N + 2 * packed, "flops": 6 * M * N}
        return {"bytes": 8 * M * N + 2 * packed, "flops": 16 * M * N}
    H, I, E, k = (case[n] for n in ("H", "I", "E", "k"))
    read = E * (1.0 - (1.0 - k / E) ** M)
    return {"bytes": 2 * (3 * H * I * read + E * H + 2 * M * H) + 4 * M * k, "flops": 2 * M * H * (E + 3 * I * k)}


def exact(case, seed):
    """The same outputs from the definitions in FP64."""
    st = prepare(case, seed)
    D = lambda n: st[n].double()  # noqa: E731
    if case["op"] in ("norm_fwd", "norm_bwd"):
        H, y = case["H"], D("y")
        gate = torch.ones_like(D("w_post")) if st["gate"] is None else D("gate")
        if case["op"] == "norm_fwd":
            r_y = (y.square().sum(1) / H + EPS).pow(-0.5)
            z = case["alpha"] * D("res") + gate * torch.einsum("mh,m,h->mh", y, r_y, D("w_post"))
            r_z = (z.square().sum(1) / H + EPS).pow(-0.5)
            return {"z": z, "h": torch.einsum("mh,m,h->mh", z, r_z, D("w_next")), "rstd": torch.stack((r_y, r_z), 1)}
        z, dh, (r_y, r_z) = D("z"), D("dh"), D("rstd").unbind(1)
        # each norm's Jacobian is r (I - n n^T / H) with n the normed row
        ny, nz = y * r_y[:, None], z * r_z[:, None]
        G = D("dz") + _project(dh * D("w_next"), nz, H) * r_z[:, None]
        dn = G * gate * D("w_post")
        dgate = G * ny * D("w_post")
        out = {"dres": case["alpha"] * G, "dy": _project(dn, ny, H) * r_y[:, None],
               "dw_post": (G * gate * ny).sum(0), "dw_next": (dh * nz).sum(0)}
        if case["gate"] != "none":
            out["dgate"] = dgate.sum(0) if case["gate"] == "row" else dgate
        return out
    if case["op"] == "ckpt8":
        g, N = D("g"), case["N"]
        top = torch.stack([c.abs().amax(1) for c in g.split(BLOCK, 1)], 1)
        s = (top / 127).repeat_interleave(BLOCK, 1)[:, :N]
        return torch.where(s > 0, torch.round(g / s) * s, 0.0)
    if case["op"] == "act8":
        g, u = (c.double() * s.double().repeat_interleave(BLOCK, 1)[:, :case["N"]] for c, s in (st["g8"], st["u8"]))
        sg = torch.sigmoid(g)
        return {"dg": D("da") * u * sg * (1 + g - g * sg), "du": D("da") * g * sg, "a": u * g * sg}
    M, H, k, E = (case[n] for n in ("M", "H", "k", "E"))
    x = D("x")
    logits = x @ D("w_router").T
    top, ids = torch.topk(logits, k, dim=1)
    p = torch.exp(top - torch.logsumexp(top if case["renorm"] else logits, 1, keepdim=True))
    y = torch.zeros(M, H, dtype=torch.float64, device=x.device)
    for e in ids.unique().tolist():
        m, j = torch.nonzero(ids == e, as_tuple=True)
        g = x[m] @ st["w_gate"][e].double().T
        a = torch.nn.functional.silu(g) * (x[m] @ st["w_up"][e].double().T)
        y.index_add_(0, m, p[m, j][:, None] * (a @ st["w_down"][e].double().T))
    return {"y": y, "p": p}


def _project(d, n, H):
    return d - n * ((d * n).sum(1, keepdim=True) / H)

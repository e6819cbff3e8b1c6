"""The operators of a mixture-of-experts training step and of 4-bit serving, as a benchmark calls them.

Five families: matrix products grouped by expert over ragged rows (grouped), the
routing of tokens to experts and its gradient (route), the weighted sum of the
experts' outputs and its gradient (combine), dropout from a counter-based
generator with the residual (dropout), and products with 4-bit weights and group
scales for a few tokens (w4).  `own` selects the library's calls; otherwise the
same operators in elementary torch operations in FP32, rounded once at the end.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def listed():
    return [
        # training step of 4096 tokens, eight of many small experts: the gate (or up) product over the sorted rows
        {"name": "grouped_nt_e128", "op": "grouped", "layout": "NT", "T": 4096, "R": 32768, "M": 0, "N": 768, "K": 2048,
         "E": 128, "empty": 0, "pair": False, "dtype": "bf16"},
        # the same tokens, two of a few experts of the dense FFN's size: the input's gradient, gate and up lanes in one sum
        {"name": "grouped_nn_e8", "op": "grouped", "layout": "NN", "T": 8192, "R": 8192, "M": 0, "N": 4096, "K": 12288,
         "E": 8, "empty": 0, "pair": True, "dtype": "bf16"},
        # the many small experts' weight gradients
        {"name": "grouped_tn_e128", "op": "grouped", "layout": "TN", "T": 4096, "R": 32768, "M": 768, "N": 2048, "K": 0,
         "E": 128, "empty": 0, "pair": False, "dtype": "bf16"},
        # a short prompt over odd sizes, experts without a token among them, FP16
        {"name": "grouped_nt_odd", "op": "grouped", "layout": "NT", "T": 127, "R": 508, "M": 0, "N": 1411, "K": 1003,
         "E": 60, "empty": 7, "pair": False, "dtype": "fp16"},
        # the training step's routing
        {"name": "route_4096_e128k8", "op": "route", "back": False, "M": 4096, "E": 128, "k": 8, "renorm": True,
         "masked": 0.0, "dtype": "fp32"},
        # the router's gradient, weights of the whole softmax, a padded batch and closed experts, 16-bit logits
        {"name": "route_bwd_777_e60k4", "op": "route", "back": True, "M": 777, "E": 60, "k": 4, "renorm": False,
         "masked": 0.1, "dtype": "bf16"},
        # the training step's experts back to tokens
        {"name": "combine_4096x2048k8", "op": "combine", "back": False, "M": 4096, "H": 2048, "k": 8, "dtype": "bf16"},
        # its gradient, towards the experts' outputs and the routing weights
        {"name": "combine_bwd_4096x2048k8", "op": "combine", "back": True, "M": 4096, "H": 2048, "k": 8, "dtype": "bf16"},
        # dropout of a block's output onto the residual, 8 sequences of 512
        {"name": "dropout_4096x4096", "op": "dropout", "M": 4096, "H": 4096, "p": 0.1, "res": True, "alpha": 1.0,
         "dtype": "bf16"},
        # its gradient at odd sizes, FP16
        {"name": "dropout_1003x5125", "op": "dropout", "M": 1003, "H": 5125, "p": 0.25, "res": False, "alpha": 1.0,
         "dtype": "fp16"},
        # serving one token through the FFN with 4-bit weights: the weights' bytes and little else
        {"name": "w4_ffn_1", "op": "w4", "ffn": True, "M": 1, "H": 4096, "I": 12288, "group": 64, "dtype": "bf16"},
        # a serving batch of 32
        {"name": "w4_ffn_32", "op": "w4", "ffn": True, "M": 32, "H": 4096, "I": 12288, "group": 64, "dtype": "bf16"},
    ]


def _log(rng, lo, hi):
    hi = max(lo, hi)
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["grouped", "grouped", "route", "combine", "dropout", "w4"])
    dtype = rng.choice(["bf16", "fp16"])
    if op == "grouped":
        layout = rng.choice(["NT", "NN", "TN"])
        E = _log(rng, 1, 256)
        a, b = _log(rng, 16, 12288), _log(rng, 16, 8192)
        if E * a * b > 1 << 29:
            b = max(16, (1 << 29) // (E * a))
        R = _log(rng, 1, min(65536, (1 << 38) // (a * b)))
        k = rng.choice([1, 2, 4, 8])
        c = {"op": op, "layout": layout, "T": max(1, R // k), "R": R, "E": E, "empty": rng.randrange((E + 3) // 4),
             "pair": layout == "NN" and rng.random() < 0.5, "dtype": dtype}
        c.update({"M": a, "N": b, "K": 0} if layout == "TN" else {"M": 0, "N": a, "K": b})
        return c
    if op == "route":
        k = rng.choice([1, 2, 4, 8])
        E = max(2 * k, _log(rng, 4, 512))
        return {"op": op, "back": rng.random() < 0.5, "M": _log(rng, 1, min(65536, (1 << 24) // E)), "E": E, "k": k,
                "renorm": rng.random() < 0.5, "masked": rng.choice([0.0, 0.1]), "dtype": rng.choice(list(DTYPES))}
    if op == "combine":
        k = rng.choice([1, 2, 4, 8])
        H = _log(rng, 64, 8192)
        return {"op": op, "back": rng.random() < 0.5, "M": _log(rng, 1, min(16384, (1 << 26) // (H * k))), "H": H, "k": k,
                "dtype": dtype}
    if op == "dropout":
        H = _log(rng, 64, 16384)
        return {"op": op, "M": _log(rng, 1, min(16384, (1 << 24) // H)), "H": H, "p": rng.choice([0.05, 0.1, 0.25, 0.5]),
                "res": rng.random() < 0.5, "alpha": rng.choice([1.0, 0.5]), "dtype": dtype}
    H = _log(rng, 64, 8192)
    I = _log(rng, 64, min(28672, (1 << 26) // H))
    return {"op": op, "ffn": rng.random() < 0.5, "M": _log(rng, 1, 128), "H": H, "I": I, "group": rng.choice([32, 64, 128]),
            "dtype": dtype}


def _rows(gen, shape, dtype, scale=1.0, shift=0.0):
    """Normal values, row-major with a leading dimension that is a multiple of 8 elements."""
    *lead, cols = shape
    buf = torch.empty((*lead, -(-cols // 8) * 8), dtype=dtype, device="cuda")
    buf.normal_(shift, scale, generator=gen)
    return buf[..., :cols]


def _int32(values):
    return torch.from_numpy(np.ascontiguousarray(values, dtype=np.int32)).cuda()


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    host = np.random.default_rng(seed)
    dt = DTYPES[case["dtype"]]
    st = {"case": case, "dtype": dt}
    op = case["op"]
    if op == "grouped":
        T, R, M, N, K, E = (case[n] for n in ("T", "R", "M", "N", "K", "E"))
        # rows an expert gets: uneven, as a router leaves them, some experts without any
        share = np.exp(host.normal(0.0, 0.5, E))
        share[host.permutation(E)[:case["empty"]]] = 0.0
        counts = host.multinomial(R, share / share.sum())
        st["host_offsets"], st["most"] = [0, *np.cumsum(counts).tolist()], int(counts.max())
        st["offsets"] = _int32(st["host_offsets"])
        # which token a row belongs to; rows in the tokens' own order need no list
        st["rows"] = _int32(host.permutation(R) % T) if T < R else None
        if case["layout"] == "TN":
            st["A"], st["B"] = _rows(gen, (R, M), dt, 0.1), _rows(gen, (T, N), dt)
        else:
            def weights():
                return _rows(gen, (E, N, K) if case["layout"] == "NT" else (E, K, N), dt, 1.0 / math.sqrt(K))
            st["A"], st["B"] = _rows(gen, (T, K), dt), weights()
            st["add"] = (_rows(gen, (T, K), dt), weights()) if case["pair"] else None
    elif op == "route":
        M, E, k = (case[n] for n in ("M", "E", "k"))
        logits = _rows(gen, (M, E), dt, 1.5)
        if case["masked"]:  # padding at the end of the batch, and experts closed to everyone
            logits[M - int(M * case["masked"]):] = -math.inf
            logits[:, torch.from_numpy(host.permutation(E)[:int(E * case["masked"])]).cuda()] = -math.inf
        st["logits"] = logits
        if case["back"]:  # what the forward left
            st["plan"] = _route_plain(logits, k, case["renorm"])
            st["dprobs"] = torch.empty((M, k), device="cuda").normal_(0.0, 0.1, generator=gen)
    elif op == "combine":
        M, H, k = (case[n] for n in ("M", "H", "k"))
        st["o"] = _rows(gen, (M * k, H), dt)
        st["pos"] = _int32(host.permutation(M * k).reshape(M, k))
        st["probs"] = torch.softmax(torch.empty((M, k), device="cuda").normal_(0.0, 1.0, generator=gen), 1)
        st["dy"] = _rows(gen, (M, H), dt, 0.1)
    elif op == "dropout":
        M, H = case["M"], case["H"]
        st["x"] = _rows(gen, (M, H), dt)
        st["res"] = _rows(gen, (M, H), dt, 1.5) if case["res"] else None
        st["rng"] = torch.tensor([int(host.integers(1 << 62)), int(host.integers(1 << 40))], device="cuda")
    else:
        M, H, I, G = (case[n] for n in ("M", "H", "I", "group"))
        st["x"] = _rows(gen, (M, H), dt)
        shapes = [(I, H), (I, H), (H, I)] if case["ffn"] else [(I, H)]
        w = [_rows(gen, s, dt, 1.0 / math.sqrt(s[1])) for s in shapes]
        if own:
            from deterministic_gated_ffn_amd import binding as dgf
            st["packed"] = [dgf.pack4(t, group=G) for t in w]
        else:
            st["packed"] = [_quantise4(t, G) for t in w]
    return st


def _route_plain(logits, k, renorm):
    """Routing by definition: ids, probs [M, k]; offsets [E + 1]; rows [M k] the token of each sorted row; pos [M, k]."""
    M, E = logits.shape
    l = torch.nan_to_num(logits.float(), nan=-math.inf, posinf=torch.finfo(torch.float32).max, neginf=-math.inf)
    top, ids = torch.sort(l, dim=1, descending=True, stable=True)
    top, ids = top[:, :k], ids[:, :k]
    taken = top > -math.inf
    e = torch.where(taken, torch.exp(top - top[:, :1]), 0.0)
    if renorm:
        den = e.sum(1, keepdim=True)
    else:
        den = torch.where(l > -math.inf, torch.exp(l - top[:, :1]), 0.0).sum(1, keepdim=True)
    probs = torch.where(taken, e / den, 0.0)
    ids = torch.where(taken, ids, -1)
    key = torch.where(taken, ids, E).reshape(-1)
    _, order = torch.sort(key, stable=True)
    offsets = torch.searchsorted(key[order], torch.arange(E + 1, device=l.device))
    live = torch.arange(M * k, device=l.device) < offsets[-1]
    rows = torch.where(live, order // k, -1)
    pos = torch.empty_like(order)
    pos[order] = torch.where(live, torch.arange(M * k, device=l.device), -1)
    i32 = torch.int32
    return {"ids": ids.to(i32), "probs": probs, "offsets": offsets.to(i32), "rows": rows.to(i32), "pos": pos.view(M, k).to(i32)}


def _quantise4(w, G):
    """(codes + 8, two a byte [N, ceil(K/2)], the lower column in the lower four bits; scales [N, ceil(K/G)]):
    scale = largest magnitude / 7 in the weights' type, code = weight / scale to nearest even, -7 to 7."""
    N, K = w.shape
    ng = -(-K // G)
    b = torch.nn.functional.pad(w.float(), (0, ng * G - K)).view(N, ng, G)
    s = (b.abs().amax(2) / 7.0).to(w.dtype)
    sf = s.float()[..., None]
    q = torch.where(sf > 0, torch.round(b / sf).clamp(-7, 7), 0.0)
    q = (q + 8).to(torch.uint8).view(N, ng * G)
    q[:, K:] = 8
    return (q[:, 0::2] | q[:, 1::2] << 4).contiguous(), s, (N, K), G


def _values4(p):
    codes, s, (N, K), G = p
    q = torch.stack((codes & 15, codes >> 4), 2).view(N, -1, G).float() - 8.0
    return (q * s.float()[..., None]).view(N, -1)[:, :K]


def run(st):
    return (_own if own else _plain)(st)


def _own(st):
    from deterministic_gated_ffn_amd import binding as dgf
    case, op = st["case"], st["case"]["op"]
    if op == "grouped":
        return dgf.gemm_grouped(case["layout"], st["A"], st["B"], st["offsets"], rows=st["rows"], add=st.get("add"))
    if op == "route":
        if case["back"]:
            return dgf.moe_route_bwd(st["dprobs"], st["logits"], st["plan"]["ids"], st["plan"]["probs"], renorm=case["renorm"])
        return dgf.moe_route(st["logits"], case["k"], renorm=case["renorm"])._asdict()
    if op == "combine":
        if case["back"]:
            do, dprobs = dgf.moe_combine_bwd(st["dy"], st["o"], st["pos"], st["probs"])
            return {"do": do, "dprobs": dprobs}
        return dgf.moe_combine(st["o"], st["pos"], st["probs"])
    if op == "dropout":
        return dgf.dropout(st["x"], case["p"], st["rng"], res=st["res"], alpha=case["alpha"])
    return (dgf.ffn_fwd_w4 if case["ffn"] else dgf.gemm_w4)(st["x"], *st["packed"])


def _plain(st):
    case, dt, op = st["case"], st["dtype"], st["case"]["op"]
    if op == "grouped":
        # every expert's rows padded with zeros to the longest one's: one batched product
        off, most, E, R = st["offsets"].long(), st["most"], case["E"], case["R"]
        at = off[:-1, None] + torch.arange(most, device="cuda")
        inside = (at < off[1:, None]).view(-1, 1)
        at = at.view(-1).clamp(max=R - 1)
        token = at if st["rows"] is None else st["rows"].long()[at]

        def padded(t, index):
            return (t[index].float() * inside).view(E, most, -1)

        if case["layout"] == "TN":
            return torch.bmm(padded(st["A"], at).transpose(1, 2), padded(st["B"], token)).to(dt)
        r = torch.arange(R, device="cuda")
        e = torch.searchsorted(off[1:], r, right=True)
        r = e * most + (r - off[e])
        c = 0.0
        for A, B in (st["A"], st["B"]), *([st["add"]] if case["pair"] else []):
            c = c + torch.bmm(padded(A, token), B.float().transpose(1, 2) if case["layout"] == "NT" else B.float())
        return c.view(E * most, -1)[r].to(dt)
    if op == "route":
        if not case["back"]:
            return _route_plain(st["logits"], case["k"], case["renorm"])
        ids, probs, dp = st["plan"]["ids"], st["plan"]["probs"], st["dprobs"]
        E = case["E"]
        s = (dp * probs).sum(1, keepdim=True)
        if case["renorm"]:
            dl = torch.zeros((case["M"], E + 1), device=dp.device)
            chosen = probs * (dp - s)
        else:
            l = st["logits"].float()
            e = torch.where(l > -math.inf, torch.exp(l - l.amax(1, keepdim=True)), 0.0)
            dl = torch.nn.functional.pad(-s * torch.where(e > 0, e / e.sum(1, keepdim=True), 0.0), (0, 1))
            chosen = probs * dp
        dl.scatter_add_(1, torch.where(ids >= 0, ids, E).long(), chosen)
        return dl[:, :E].to(dt)
    if op == "combine":
        M, H, k = (case[n] for n in ("M", "H", "k"))
        o = st["o"][st["pos"].view(-1)].float().view(M, k, H)
        if not case["back"]:
            return (o * st["probs"][:, :, None]).sum(1).to(dt)
        dy = st["dy"].float()[:, None]
        do = torch.empty((M * k, H), dtype=dt, device=o.device)
        do[st["pos"].view(-1)] = (dy * st["probs"][:, :, None]).to(dt).view(M * k, H)
        return {"do": do, "dprobs": (dy * o).sum(2)}
    if op == "dropout":
        M, H = case["M"], case["H"]
        cut = int(round(case["p"] * 65536))
        seed, step = st["rng"][0], st["rng"][1]
        low = 0xFFFFFFFF
        n = M * -(-H // 8)
        i = torch.arange(n, device="cuda")
        c = [i & low, i >> 32, (step & low).expand(n), ((step >> 32) & low).expand(n)]
        k0, k1 = seed & low, (seed >> 32) & low
        for r in range(10):  # Philox-4x32-10: two 32 x 32 -> 64-bit products a round
            a, b = c[0] * 0xD2511F53, c[2] * 0xCD9E8D57
            c = [(b >> 32 & low) ^ c[1] ^ k0, b & low, (a >> 32 & low) ^ c[3] ^ k1, a & low]
            k0, k1 = (k0 + 0x9E3779B9) & low, (k1 + 0xBB67AE85) & low
        draws = torch.stack([h for w in c for h in (w & 0xFFFF, w >> 16)], 1).view(M, -1)[:, :H]
        z = torch.where(draws >= cut, st["x"].float() * (65536.0 / (65536 - cut)), 0.0)
        return (z if st["res"] is None else case["alpha"] * st["res"].float() + z).to(dt)
    x, w = st["x"].float(), [_values4(p) for p in st["packed"]]
    if not case["ffn"]:
        return (x @ w[0].t()).to(dt)
    g = x @ w[0].t()
    return ((g / (1.0 + torch.exp(-g)) * (x @ w[1].t())) @ w[2].t()).to(dt)


def work(case):
    """Bytes: each input read once (the weights of every expert that has a row), each output written once."""
    op = case["op"]
    size = 4 if case["dtype"] == "fp32" else 2
    if op == "grouped":
        T, R, M, N, K, E = (case[n] for n in ("T", "R", "M", "N", "K", "E"))
        lists = 4 * (E + 1) + (4 * R if T < R else 0)
        if case["layout"] == "TN":
            return {"bytes": 2 * (R * M + T * N + E * M * N) + lists, "flops": 2 * R * M * N}
        terms = 2 if case["pair"] else 1
        used = min(R, E - case["empty"])
        return {"bytes": 2 * (terms * (T * K + used * N * K) + R * N) + lists, "flops": 2 * terms * R * N * K}
    if op == "route":
        M, E, k = (case[n] for n in ("M", "E", "k"))
        if case["back"]:
            return {"bytes": M * E * size * (1 if case["renorm"] else 2) + 12 * M * k, "flops": 6 * M * E}
        return {"bytes": M * E * size + 16 * M * k + 4 * (E + 1), "flops": 6 * M * E}
    if op == "combine":
        M, H, k = (case[n] for n in ("M", "H", "k"))
        if case["back"]:
            return {"bytes": 2 * M * H * (2 * k + 1) + 12 * M * k, "flops": 3 * M * k * H}
        return {"bytes": 2 * M * H * (k + 1) + 8 * M * k, "flops": 2 * M * k * H}
    if op == "dropout":
        n = case["M"] * case["H"]
        return {"bytes": 2 * n * (3 if case["res"] else 2), "flops": 12 * n}
    M, H, I, G = (case[n] for n in ("M", "H", "I", "group"))
    w = I * -(-H // 2) + 2 * I * -(-H // G)
    if not case["ffn"]:
        return {"bytes": w + 2 * M * (H + I), "flops": 2 * M * H * I}
    return {"bytes": 2 * w + H * -(-I // 2) + 2 * H * -(-I // G) + 4 * M * H, "flops": 6 * M * H * I}


def exact(case, seed):
    """The same outputs from the definitions in FP64."""
    st = prepare(case, seed)
    op = case["op"]
    D = lambda n: st[n].double()  # noqa: E731
    if op == "grouped":
        off = st["host_offsets"]
        where = torch.arange(case["R"], device="cuda") if st["rows"] is None else st["rows"].long()
        if case["layout"] == "TN":
            out = torch.zeros(case["E"], case["M"], case["N"], dtype=torch.float64, device="cuda")
            for e in range(case["E"]):
                r = slice(off[e], off[e + 1])
                out[e] = torch.mm(D("A")[r].T, st["B"][where[r]].double())
            return out
        out = torch.zeros(case["R"], case["N"], dtype=torch.float64, device="cuda")
        for A, B in [(st["A"], st["B"])] + ([st["add"]] if st["add"] else []):
            for e in range(case["E"]):
                r = slice(off[e], off[e + 1])
                w = B[e].double()
                out[r] += torch.mm(A[where[r]].double(), w.T if case["layout"] == "NT" else w)
        return out
    if op == "route":
        return _route_exact(st)
    if op == "combine":
        pos = st["pos"].long()
        if not case["back"]:
            y = torch.zeros(case["M"], case["H"], dtype=torch.float64, device="cuda")
            for j in range(case["k"]):
                y += D("probs")[:, j, None] * D("o")[pos[:, j]]
            return y
        do = torch.zeros(case["M"] * case["k"], case["H"], dtype=torch.float64, device="cuda")
        dprobs = torch.zeros(case["M"], case["k"], dtype=torch.float64, device="cuda")
        for j in range(case["k"]):
            do[pos[:, j]] = D("probs")[:, j, None] * D("dy")
            dprobs[:, j] = torch.linalg.vecdot(D("dy"), D("o")[pos[:, j]])
        return {"do": do, "dprobs": dprobs}
    if op == "dropout":
        M, H = case["M"], case["H"]
        cut = int(round(case["p"] * 65536))
        keep = torch.from_numpy(_philox_halves(*st["rng"].tolist(), M * -(-H // 8)).reshape(M, -1)[:, :H] >= cut).cuda()
        z = D("x") * keep * (65536 / (65536 - cut))
        return z if st["res"] is None else z + case["alpha"] * D("res")
    w = []
    for codes, s, (N, K), G in st["packed"]:
        q = torch.empty(N, 2 * codes.shape[1], dtype=torch.float64, device="cuda")
        q[:, 0::2], q[:, 1::2] = (codes % 16).double(), (codes // 16).double()
        w.append(((q - 8) * s.double().repeat_interleave(G, 1))[:, :K])
    x = D("x")
    if not case["ffn"]:
        return x @ w[0].T
    return (torch.nn.functional.silu(x @ w[0].T) * (x @ w[1].T)) @ w[2].T


def _route_exact(st):
    case = st["case"]
    M, E, k = (case[n] for n in ("M", "E", "k"))
    l = st["logits"].double().cpu().numpy()
    whole = np.exp(l - np.maximum(l.max(1, keepdims=True), -1e300))
    if case["back"]:
        ids, p, dp = (st[a][b].double().cpu().numpy() if b else st[a].double().cpu().numpy()
                      for a, b in (("plan", "ids"), ("plan", "probs"), ("dprobs", None)))
        g = np.zeros((M, E + 1))  # the loss's gradient at each expert's weight
        g[np.arange(M)[:, None], ids.astype(int)] = dp
        if case["renorm"]:
            P = np.zeros((M, E + 1))
            P[np.arange(M)[:, None], ids.astype(int)] = p
            P[:, E] = 0.0
        else:
            total = whole.sum(1, keepdims=True)
            P = np.pad(np.divide(whole, total, out=np.zeros_like(whole), where=total > 0), ((0, 0), (0, 1)))
        g, P = g[:, :E], P[:, :E]
        return torch.from_numpy(P * (g - (P * g).sum(1, keepdims=True))).cuda()
    ids = np.argsort(-l, axis=1, kind="stable")[:, :k]
    live = np.take_along_axis(l, ids, 1) > -np.inf
    p = np.where(live, np.take_along_axis(whole, ids, 1), 0.0)
    den = p.sum(1, keepdims=True) if case["renorm"] else whole.sum(1, keepdims=True)
    p = np.divide(p, den, out=np.zeros_like(p), where=den > 0)
    ids = np.where(live, ids, -1)
    lists = [[] for _ in range(E)]
    for n, e in enumerate(ids.reshape(-1).tolist()):
        if e >= 0:
            lists[e].append(n)
    order = np.array([n for one in lists for n in one], dtype=np.int64)
    rows, pos = np.full(M * k, -1), np.full(M * k, -1)
    rows[:len(order)] = order // k
    pos[order] = np.arange(len(order))
    offsets = np.cumsum([0] + [len(one) for one in lists])
    out = {"ids": ids, "probs": p, "offsets": offsets, "rows": rows, "pos": pos.reshape(M, k)}
    return {n: torch.from_numpy(v if n == "probs" else v.astype(np.int32)).cuda() for n, v in out.items()}


def _philox_halves(seed, step, n):
    """The 16-bit halves of n blocks of the generator, [n, 8], low half first."""
    u = np.uint64
    low, sh = u(0xFFFFFFFF), u(32)
    i = np.arange(n, dtype=u)
    ctr = [i & low, i >> sh, np.full(n, step & 0xFFFFFFFF, u), np.full(n, step >> 32 & 0xFFFFFFFF, u)]
    key = [seed & 0xFFFFFFFF, seed >> 32 & 0xFFFFFFFF]
    for _ in range(10):
        first, second = ctr[0] * u(0xD2511F53), ctr[2] * u(0xCD9E8D57)
        ctr = [(second >> sh) ^ ctr[1] ^ u(key[0]), second & low, (first >> sh) ^ ctr[3] ^ u(key[1]), first & low]
        key = [(key[0] + 0x9E3779B9) & 0xFFFFFFFF, (key[1] + 0xBB67AE85) & 0xFFFFFFFF]
    out = np.empty((n, 8), dtype=np.int32)
    for j, word in enumerate(ctr):
        out[:, 2 * j], out[:, 2 * j + 1] = word & u(0xFFFF), word >> u(16)
    return out

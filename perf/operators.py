"""Cases for the operators around the 4-bit products of a decoder layer: the
router of a mixture-of-experts layer, the whole layer on tiled 4-bit experts,
the 8-bit block quantizer, and the product of 8-bit block-scaled matrices.

``run`` computes each operator in elementary torch operations (32 bits, or 64
where a selection hangs on the value) or, with ``own``, through the package.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
Q8 = torch.float8_e4m3fn


def listed():
    return [
        # one token through a router of many small experts: pure latency
        dict(name="route_1x64", op="route", T=1, H=2048, E=64, k=6, x="bf16", mode="softmax"),
        # a decode batch through sigmoid scores with a selection bias
        dict(name="route_48x256", op="route", T=48, H=4096, E=256, k=8, x="f16", mode="sigmoid"),
        # single-token decode, many small experts
        dict(name="moe_q4_0_1x64e", op="moe", fmt="q4_0", T=1, H=2048, I=1408, E=64, k=6, x="f16",
             y="f16", mode="norm"),
        # single-token decode, two of eight experts of the dense layer's size
        dict(name="moe_q4_0_1x8e", op="moe", fmt="q4_0", T=1, H=4096, I=11008, E=8, k=2, x="bf16",
             y="bf16", mode="norm"),
        # a few tokens (speculative decode), super-block experts, fp32 residual stream
        dict(name="moe_ksb_5x32e", op="moe", fmt="ksb", T=5, H=4096, I=1536, E=32, k=4, x="f32",
             y="f32", mode="softmax"),
        # a decode batch that touches nearly every expert
        dict(name="moe_q4_0_32x64e", op="moe", fmt="q4_0", T=32, H=2048, I=1408, E=64, k=6,
             x="bf16", y="bf16", mode="sigmoid"),
        # activations of a short batch, and a whole weight matrix when a model is loaded
        dict(name="quant_rows_7x4096", op="quant", R=7, K=4096, rows=1, x="bf16"),
        dict(name="quant_tiles_11008x4096", op="quant", R=11008, K=4096, rows=128, x="f32"),
        # decode, a ragged batch, a prompt, a long prompt
        dict(name="fp8_1x4096x4096", op="gemm", B=1, M=4096, K=4096, y="bf16"),
        dict(name="fp8_37x11000x4096", op="gemm", B=37, M=11000, K=4096, y="f16"),
        dict(name="fp8_500x4096x11008", op="gemm", B=500, M=4096, K=11008, y="bf16"),
        dict(name="fp8_4096x11008x4096", op="gemm", B=4096, M=11008, K=4096, y="f32"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["route", "moe", "moe", "quant", "gemm", "gemm"])
    if op == "route":
        E = _log(rng, 4, 512)
        return dict(op=op, T=_log(rng, 1, 64), H=8 * _log(rng, 32, 1024), E=E,
                    k=rng.randint(1, min(E, 12)), x=rng.choice(list(DTYPES)),
                    mode=rng.choice(["softmax", "norm", "sigmoid"]))
    if op == "moe":
        fmt = rng.choice(["q4_0", "ksb"])
        step = 64 if fmt == "q4_0" else 256
        H, I = step * _log(rng, 512 // step, 6144 // step), step * _log(rng, 256 // step, 11008 // step)
        E = _log(rng, 2, min(256, max(3, 1_000_000_000 // (3 * H * I))))
        return dict(op=op, fmt=fmt, T=_log(rng, 1, 40), H=H, I=I, E=E, k=rng.randint(1, min(E, 8)),
                    x=rng.choice(list(DTYPES)), y=rng.choice(list(DTYPES)),
                    mode=rng.choice(["softmax", "norm", "sigmoid"]))
    if op == "quant":
        K = 16 * _log(rng, 8, 1024)
        return dict(op=op, R=_log(rng, 1, 45_000_000 // K), K=K, rows=rng.choice([1, 128]),
                    x=rng.choice(list(DTYPES)))
    M, K = _log(rng, 200, 12000), 16 * _log(rng, 16, 700)
    return dict(op=op, B=_log(rng, 1, min(8192, 180_000_000_000 // (M * K))), M=M, K=K,
                y=rng.choice(list(DTYPES)))


# ------------------------------------------------------------------- inputs
def _tiled_bytes(fmt, R, K):
    return R * (K // 32 * 18 if fmt == "q4_0" else K // 256 * 138)


def _sections(fmt, T, R, K):
    """The tiles of R x K tiled storage as byte views: [(codes, scales...)] of the full tiles and
    of the last, shorter one; each [R / 16, tiles, bytes]."""
    per = 64 if fmt == "q4_0" else 8
    nblk = K // (32 if fmt == "q4_0" else 256)
    tile = 18432 if fmt == "q4_0" else 17664
    rows = T.view(R // 16, -1)
    full, rest = nblk // per, nblk % per

    def cut(v, nb):
        if fmt == "q4_0":
            return v[..., :256 * nb], v[..., 256 * nb:]
        return v[..., :2048 * nb], v[..., 2048 * nb:2176 * nb], v[..., 2176 * nb:]

    parts = []
    if full:
        parts.append((per, cut(rows[:, :full * tile].unflatten(1, (full, tile)), per)))
    if rest:
        parts.append((rest, cut(rows[:, full * tile:].unsqueeze(1), rest)))
    return parts


def _experts(fmt, R, K, g):
    """Tiled storage of R x K weights as the quantizers leave N(0, 0.02^2) ones: bell-shaped codes,
    scales near 2.1 / 7 of the deviation."""
    T = torch.empty(_tiled_bytes(fmt, R, K), dtype=torch.uint8, device="cuda")
    for nb, sec in _sections(fmt, T, R, K):
        n = sec[0].numel()
        codes = torch.randn(2, n, device="cuda", generator=g).mul_(3.2).round_().add_(8).clamp_(1, 15)
        codes = codes.to(torch.uint8)
        sec[0].copy_((codes[0] | codes[1] << 4).view(sec[0].shape))
        u = torch.rand(sec[-1].numel() // 2, device="cuda", generator=g)
        if fmt == "q4_0":
            d = 0.006 * (0.6 + 0.8 * u)
        else:  # INT8 sub-scales up to 127 against one fp16 scale
            q = torch.randint(40, 128, (sec[1].numel(),), device="cuda", generator=g)
            sec[1].copy_(q.to(torch.uint8).view(sec[1].shape))
            d = 0.006 / 90 * (0.6 + 0.8 * u)
        sec[-1].copy_(d.to(torch.float16).view(torch.uint8).view(sec[-1].shape))
    return T


def _fp8(R, K, rows, g, std):
    """A matrix in 8-bit blocks as the quantizer leaves it: codes over the whole range, scales of
    blocks that differ."""
    v = torch.randn(R, K, device="cuda", generator=g).mul_(120.0).clamp_(-448, 448)
    s = torch.rand((R + rows - 1) // rows, (K + 127) // 128, device="cuda", generator=g)
    return v.to(Q8), (std / 120) * torch.exp(1.2 * (s - 0.5))


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    op, st = case["op"], dict(case)
    rand = lambda *n: torch.randn(*n, device="cuda", generator=g)  # noqa: E731
    if op in ("route", "moe"):
        T, H, E = case["T"], case["H"], case["E"]
        st["xs"] = rand(T, H).to(DTYPES[case["x"]])
        st["Wr"] = (rand(E, H) / math.sqrt(H)).to(torch.bfloat16)
        # a bias balances the load of sigmoid routers
        st["bias"] = 0.05 * rand(E) if case["mode"] == "sigmoid" else None
    if op == "moe":
        fmt, H, I, E = case["fmt"], case["H"], case["I"], case["E"]
        st["gate"], st["up"] = _experts(fmt, E * I, H, g), _experts(fmt, E * I, H, g)
        st["down"] = _experts(fmt, E * H, I, g)
    if op == "quant":
        x = rand(case["R"], case["K"])
        x *= torch.exp(2 * rand(case["R"], 1)) if case["rows"] == 1 else 0.02
        st["xs"] = x.to(DTYPES[case["x"]])
    if op == "gemm":
        st["W"], st["ws"] = _fp8(case["M"], case["K"], 128, g, 0.02)
        st["X"], st["xsc"] = _fp8(case["B"], case["K"], 1, g, 1.0)
    return st


# -------------------------------------------------------------- plain forms
def _decode(fmt, T, n, R, K):
    """n matrices of R x K tiled weights (bytes [n, ...]) in 32 bits, [n, R, K]."""
    cols = []
    for nb, sec in _sections(fmt, T.reshape(-1), n * R, K):
        G, c = sec[0].shape[:2]
        units = nb // 2 if fmt == "q4_0" else 2 * nb
        blocks = 2 if fmt == "q4_0" else 4  # blocks of 32 weights in a unit
        # [group, tile, unit, row % 8, word, block, row / 8, byte]
        q = sec[0].reshape(G, c, units, 8, 4, blocks, 2, 4)
        w = torch.stack((q & 15, q >> 4), dim=6).float() - 8.0
        # -> [group, row / 8, row % 8, tile, unit, block, nibble, word, byte]
        w = w.permute(0, 7, 3, 1, 2, 5, 6, 4, 8)
        if fmt == "q4_0":
            d = sec[1].contiguous().view(torch.float16).float().view(G, c, units, 16, 2)
            s = d.permute(0, 3, 1, 2, 4)
        else:
            q8 = sec[1].contiguous().view(torch.int8).float().view(G, c, nb, 2, 16, 4)
            S = sec[2].contiguous().view(torch.float16).float().view(G, c, nb, 1, 16, 1)
            s = (S * q8).permute(0, 4, 1, 2, 3, 5)
        w = w.reshape(G, 16, c * units * blocks, 32) * s.reshape(G, 16, c * units * blocks, 1)
        cols.append(w.reshape(n, R, -1))
    return torch.cat(cols, dim=2)


def _route(st):
    # in 64 bits: which experts are taken hangs on values next to each other
    logits = st["xs"].double() @ st["Wr"].double().T
    if st["mode"] == "sigmoid":
        score = torch.sigmoid(logits)
        key = score + st["bias"].double()
    else:
        score, key = torch.softmax(logits, dim=1), logits
    ids = torch.sort(key, dim=1, descending=True, stable=True).indices[:, :st["k"]]
    w = score.gather(1, ids)
    if st["mode"] != "softmax":
        w = w / w.sum(dim=1, keepdim=True)
    return ids.to(torch.int32), w.float()


def _moe(st):
    ids, w = _route(st)
    fmt, T, H, I, E, k = (st[n] for n in ("fmt", "T", "H", "I", "E", "k"))
    x = st["xs"].float()
    gate, up, down = st["gate"].view(E, -1), st["up"].view(E, -1), st["down"].view(E, -1)
    if T * k < E:  # the chosen experts' matrices alone
        pick = ids.reshape(-1).long()
        xe = x.repeat_interleave(k, dim=0).unsqueeze(2)
        mix = w.view(T, k, 1)
        n = T * k
        gate, up, down = gate[pick], up[pick], down[pick]
    else:  # every expert on every token
        xe = x.T.expand(E, H, T)
        mix = torch.zeros(T, E, device=x.device).scatter_add_(1, ids.long(), w).T.reshape(E, 1, T)
        n = E
    a = torch.bmm(_decode(fmt, gate, n, I, H), xe)
    b = torch.bmm(_decode(fmt, up, n, I, H), xe)
    o = torch.bmm(_decode(fmt, down, n, H, I), a / (1 + torch.exp(-a)) * b)
    y = (o.view(T, k, H) * mix).sum(dim=1) if T * k < E else (o * mix).sum(dim=0).T
    return y.to(DTYPES[st["y"]])


def _blocks(x, rows):
    """x padded with zeros to whole blocks: [row blocks, rows, column blocks, 128]."""
    R, K = x.shape
    x = torch.nn.functional.pad(x, (0, -K % 128, 0, -R % rows))
    return x.view(x.shape[0] // rows, rows, x.shape[1] // 128, 128)


def _spread(s, rows, R, K):
    return s.repeat_interleave(rows, dim=0)[:R].repeat_interleave(128, dim=1)[:, :K]


def _quant(st):
    x, rows = st["xs"].float(), st["rows"]
    R, K = x.shape
    # a tensor as divisor: by a number, torch multiplies by its reciprocal
    scale = _blocks(x, rows).abs().amax(dim=(1, 3)) / torch.full((), 448.0, device=x.device)
    q = torch.where(_spread(scale, rows, R, K) > 0, x / _spread(scale, rows, R, K), 0.0)
    return q.clamp(-448, 448).to(Q8), scale


def _gemm(st):
    W = st["W"].float() * _spread(st["ws"], 128, *st["W"].shape)
    X = st["X"].float() * _spread(st["xsc"], 1, *st["X"].shape)
    return (X @ W.T).to(DTYPES[st["y"]])


def _own(st):
    import bit_gemv_q4_b200 as gq
    op = st["op"]
    if op in ("route", "moe"):
        flags = {"softmax": 0, "norm": gq.GQ_ROUTE_NORM,
                 "sigmoid": gq.GQ_ROUTE_SIGMOID | gq.GQ_ROUTE_NORM}[st["mode"]]
        ids, w = gq.gq_moe_route(st["xs"], st["Wr"], st["k"], bias=st["bias"], flags=flags)
        if op == "route":
            return ids, w
        layer = gq.gq_moe_q4_0_tiled if st["fmt"] == "q4_0" else gq.gq_moe_ksb_tiled
        return layer(st["gate"], st["up"], st["down"], st["E"], st["I"], st["xs"], ids, w,
                     y_dtype=DTYPES[st["y"]], flags=gq.GQ_GEMV_PDL)
    if op == "quant":
        return gq.gq_quantize_fp8(st["xs"], st["rows"])
    return gq.gq_gemm_fp8(st["W"], st["ws"], st["X"], st["xsc"], y_dtype=DTYPES[st["y"]])


def run(state):
    if own:
        return _own(state)
    return {"route": _route, "moe": _moe, "quant": _quant, "gemm": _gemm}[state["op"]](state)


# --------------------------------------------------------------------- work
def work(case):
    size = {"f32": 4, "f16": 2, "bf16": 2}
    op = case["op"]
    if op == "route":
        T, H, E, k = (case[n] for n in ("T", "H", "E", "k"))
        return {"bytes": 2 * E * H + size[case["x"]] * T * H + 8 * T * k, "flops": 2 * T * H * E}
    if op == "moe":
        T, H, I, E, k = (case[n] for n in ("T", "H", "I", "E", "k"))
        taken = E * (1 - (1 - k / E) ** T)  # experts that some token takes, on average
        return {"bytes": 2 * E * H + taken * 3 * _tiled_bytes(case["fmt"], H, I)
                + T * H * (size[case["x"]] + size[case["y"]]),
                "flops": 2 * T * H * E + 6 * T * k * H * I}
    if op == "quant":
        R, K = case["R"], case["K"]
        blocks = -(-R // case["rows"]) * -(-K // 128)
        return {"bytes": R * K * (size[case["x"]] + 1) + 4 * blocks, "flops": 3 * R * K}
    B, M, K = case["B"], case["M"], case["K"]
    kb = -(-K // 128)
    return {"bytes": (M + B) * K + 4 * kb * (B + -(-M // 128)) + B * M * size[case["y"]],
            "flops": 2 * B * M * K}


# ---------------------------------------------------------- in 64 bits, apart
def _weights64(fmt, T, R, K, expert):
    """Expert `expert` of tiled storage, weight by weight: the byte offset of each code and scale
    from the layout's definition."""
    r = torch.arange(expert * R, (expert + 1) * R, device=T.device).view(-1, 1)
    k = torch.arange(K, device=T.device).view(1, -1)
    g, r = r // 16, r % 16
    hi, wt, lane8, half = (k % 32) // 16, (k % 16) // 4, r % 8, r // 8
    byte = k % 4
    f16 = lambda at: (T[at].int() | T[at + 1].int() << 8).to(torch.int16).view(torch.float16).double()  # noqa: E731
    if fmt == "q4_0":
        b = k // 32
        c, b = b // 64, b % 64
        nb = torch.clamp(K // 32 - 64 * c, max=64)
        tile = g * (16 * (K // 32) * 18) + c * 18432
        code = tile + 512 * (b // 2) + 16 * (4 * lane8 + wt) + 8 * (b % 2) + 4 * half + byte
        scale = f16(tile + 256 * nb + 64 * (b // 2) + 4 * r + 2 * (b % 2))
    else:
        sb, j = k // 256, k % 256 // 32
        c, sb = sb // 8, sb % 8
        ns = torch.clamp(K // 256 - 8 * c, max=8)
        tile = g * (16 * (K // 256) * 138) + c * 17664
        u = 2 * sb + j // 4
        code = tile + 1024 * u + 32 * (4 * lane8 + wt) + 8 * (j % 4) + 4 * half + byte
        sub = T[tile + 2048 * ns + 64 * u + 4 * r + j % 4].to(torch.int8).double()
        scale = f16(tile + 2176 * ns + 32 * sb + 2 * r) * sub
    return scale * ((T[code].int() >> (4 * hi)) % 16 - 8).double()


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op in ("route", "moe"):
        x, Wr, k = st["xs"].double(), st["Wr"].double(), case["k"]
        z = (x[:, None, :] * Wr[None]).sum(-1) if x.shape[0] * Wr.numel() < 1 << 28 else x.matmul(Wr.t())
        if case["mode"] == "sigmoid":
            score = 1 / (1 + torch.exp(-z))
            key = score + st["bias"].double()
        else:
            score = torch.exp(z - z.amax(1, keepdim=True))
            score = score / score.sum(1, keepdim=True)
            key = z
        ids = []
        for _ in range(k):  # the largest that is left, the first of equals
            ids.append(key.argmax(dim=1))
            key = key.scatter(1, ids[-1][:, None], -math.inf)
        ids = torch.stack(ids, 1)
        w = torch.stack([score[t, ids[t]] for t in range(len(ids))])
        if case["mode"] != "softmax":
            w = w / w.sum(1, keepdim=True)
        if op == "route":
            return ids, w
        y = torch.zeros(case["T"], case["H"], dtype=torch.float64, device="cuda")
        for e in ids.unique().tolist():
            t, j = (ids == e).nonzero(as_tuple=True)
            G = _weights64(case["fmt"], st["gate"], case["I"], case["H"], e) @ x[t].T
            U = _weights64(case["fmt"], st["up"], case["I"], case["H"], e) @ x[t].T
            D = _weights64(case["fmt"], st["down"], case["H"], case["I"], e)
            y[t] += w[t, j, None] * (D @ (G * torch.sigmoid(G) * U)).T
        return y
    if op == "quant":
        x = st["xs"].double()  # the codes round quotients in 32 bits, by definition
        top = torch.stack([c.abs().amax(dim=1) for c in x.split(128, dim=1)], dim=1)
        return None, torch.stack([r.amax(dim=0) for r in top.split(case["rows"])]) / 448
    B, M, K = case["B"], case["M"], case["K"]
    if B * M * K > 400_000_000_000:
        return None
    y = torch.zeros(B, M, dtype=torch.float64, device="cuda")
    for b in range((K + 127) // 128):
        at = slice(128 * b, min(K, 128 * b + 128))
        part = st["X"][:, at].double() @ st["W"][:, at].double().T
        y += part * st["xsc"][:, b, None].double() * st["ws"][:, b].double().repeat_interleave(128)[:M]
    return y

"""Cases of the balance loss, the 8-bit checkpoints and the 8-bit integer products, with their plain forms.

Three operators are listed here:

* the balance loss of a router with the counts of each expert, whole batch or
  sequence by sequence, and its gradient (``moe_balance``, ``moe_balance_bwd``);
* the experts' gated block that keeps gate and up values in 8 bits, and the
  backward pass that reads them (``moe_glu_keep8``, ``moe_glu_bwd_keep8``);
* products in 8-bit integers with a scale for each token and each channel: the
  cast of rows (``i8_group_cast``), a projection of any number of rows
  (``i8_linear``), the experts' products (``i8_group_gemm``, ``i8_group_glu``)
  and their forms for single tokens (``i8_token_glu``, ``i8_token_linear``).

``run`` computes them with elementary torch operations in 32 bits, or, where
``own`` is true, through the package's entry points.  ``exact`` computes them
from their definitions in 64 bits.
"""
import random

import numpy as np
import torch

own = False

DEV = "cuda"
ROW_GROUP = 128          # rows of an expert's group come in multiples of this
KEEP_GROUP = 32          # columns that share a scale of the kept values
FLT_MAX = 3.4028234663852886e38
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ------------------------------------------------------------------- cases

def listed():
    return [
        # a small batch of a test run: latency of both passes counts
        dict(name="balance_small", op="balance", T=33, E=8, k=2, dtype="f32", score="softmax", S=1, add=False),
        # a large training batch, one loss over all of its tokens
        dict(name="balance_batch", op="balance", T=32768, E=256, k=8, dtype="f32", score="softmax", S=1, add=False),
        # packed sequences of uneven length, a loss for each; the gradient joins the one of the weights
        dict(name="balance_seqs", op="balance", T=8191, E=64, k=6, dtype="bf16", score="sigmoid", S=11, add=True),
        # training step of the block on one device's share of the experts: forward that keeps 8 bits, backward on them
        dict(name="keep8_batch", op="keep8", M=16384, E=32, H=7168, F=2048, act="silu"),
        # many small experts, columns that end inside a scale's group
        dict(name="keep8_odd", op="keep8", M=8192, E=64, H=2048, F=1040, act="gelu"),
        # a decoding batch of eight rows through a dense projection
        dict(name="linear_tokens", op="linear", T=8, N=7168, K=2048, out="bf16"),
        # some hundred rows of short prompts, sizes that fill no tile
        dict(name="linear_ragged", op="linear", T=193, N=2064, K=5920, out="f32"),
        # prompts of a batch through a dense projection
        dict(name="linear_prompts", op="linear", T=4095, N=7168, K=7168, out="bf16"),
        # gate and up projection of a large batch, skewed routing over 32 experts
        dict(name="experts_glu", op="experts_glu", M=65536, E=32, H=7168, F=2048, act="silu"),
        # down projection of packed rows with spare capacity, routing from device offsets
        dict(name="experts_down", op="experts", M=32768, E=64, N=7168, K=2048, out="f32", spare=4096),
        # one decoding token: the 8 chosen experts' gate and up weights are read once
        dict(name="token_glu", op="token_glu", T=1, E=32, k=8, H=7168, F=2048, act="silu"),
        # a ragged decoding batch: several tokens meet in some experts; down projection
        dict(name="token_down", op="token_down", T=24, E=64, k=6, H=7168, F=2048),
    ]


def _log(rng, lo, hi):
    """A whole number between lo and hi, spread over its logarithm."""
    v = int(round(lo * (hi / lo) ** rng.random()))
    return max(lo, min(hi, v))


def draw(rng):
    op = rng.choice(["balance", "balance", "keep8", "linear", "linear", "experts", "experts_glu", "token_glu", "token_down"])
    if op == "balance":
        E = rng.choice([8, 16, 40, 64, 100, 128, 160, 256, 384, 512])
        T = _log(rng, 1, 32768 * 256 // E if E >= 256 else 32768)
        return dict(op=op, T=T, E=E, k=rng.randint(1, min(E, 10)), dtype=rng.choice(["f32", "bf16"]),
                    score=rng.choice(["softmax", "sigmoid"]), S=rng.choice([1, _log(rng, 1, 64)]), add=rng.random() < 0.5)
    if op == "keep8":
        return dict(op=op, M=ROW_GROUP * _log(rng, 1, 128), E=rng.choice([1, 4, 8, 16, 32, 64]), H=128 * _log(rng, 2, 56),
                    F=16 * _log(rng, 8, 128), act=rng.choice(["silu", "gelu"]))
    if op == "linear":
        return dict(op=op, T=_log(rng, 1, 8192), N=16 * _log(rng, 16, 448), K=16 * _log(rng, 16, 448),
                    out=rng.choice(["f32", "bf16"]))
    if op == "experts":
        return dict(op=op, M=ROW_GROUP * _log(rng, 1, 256), E=rng.choice([1, 4, 8, 16, 32, 64]), N=16 * _log(rng, 16, 448),
                    K=16 * _log(rng, 16, 448), out=rng.choice(["f32", "bf16"]), spare=ROW_GROUP * rng.randint(0, 16))
    if op == "experts_glu":
        return dict(op=op, M=ROW_GROUP * _log(rng, 1, 256), E=rng.choice([1, 4, 8, 16, 32, 64]), H=16 * _log(rng, 16, 448),
                    F=16 * _log(rng, 8, 128), act=rng.choice(["silu", "gelu"]))
    E = rng.choice([1, 8, 16, 32, 64])
    c = dict(op=op, T=_log(rng, 1, 64), E=E, k=rng.randint(1, min(E, 8)), H=16 * _log(rng, 16, 448), F=16 * _log(rng, 16, 128))
    if op == "token_glu":
        c["act"] = rng.choice(["silu", "gelu"])
    return c


# ------------------------------------------------------------------- inputs

def _seeded(seed, salt):
    g = torch.Generator(device=DEV)
    g.manual_seed((int(seed) * 1000003 + salt * 7919 + 29) % (1 << 62))
    return g


def _cast_nvfp4(x):
    """Row-scaled NVFP4 of f32 lines [L, K]: codes u8 [L, K/2], E4M3 bytes [L, K/16], line amax f32 [L]."""
    L, K = x.shape
    amax = x.abs().amax(1)
    s = (amax / 2688.0).clamp_min(1e-30)
    b = x.view(L, K // 16, 16)
    S = ((b.abs().amax(2) / 6.0) / s[:, None]).clamp(max=448.0).to(torch.float8_e4m3fn)
    d = S.float() * s[:, None]
    v = torch.where(d[..., None] > 0, b / d[..., None].clamp_min(1e-37), torch.zeros((), device=x.device))
    edges = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=x.device)
    code = torch.bucketize(v.abs(), edges, out_int32=True).to(torch.uint8) + 8 * (v < 0).to(torch.uint8)
    code = code.view(L, K // 2, 2)
    return (code[..., 0] | (code[..., 1] << 4)).contiguous(), S.view(torch.uint8), amax


def _rows_values(g, n, K):
    """Rows of activations: normal values times a scale of the row."""
    return torch.randn((n, K), generator=g, device=DEV) * torch.exp(0.5 * torch.randn((n, 1), generator=g, device=DEV))


def _rows_nvfp4(g, rows, K):
    data = torch.empty((rows, K // 2), dtype=torch.uint8, device=DEV)
    scale = torch.empty((rows, K // 16), dtype=torch.uint8, device=DEV)
    amax = torch.empty(rows, device=DEV)
    for i in range(0, rows, 8192):
        n = min(8192, rows - i)
        data[i:i + n], scale[i:i + n], amax[i:i + n] = _cast_nvfp4(_rows_values(g, n, K))
    return data, scale, amax


def _weights_nvfp4(g, E, N, K):
    """Weights of E experts, N lines of K each, with the spread that keeps outputs near one."""
    data = torch.empty((E, N, K // 2), dtype=torch.uint8, device=DEV)
    scale = torch.empty((E, N, K // 16), dtype=torch.uint8, device=DEV)
    amax = torch.empty((E, N), device=DEV)
    for e in range(E):
        data[e], scale[e], amax[e] = _cast_nvfp4(torch.randn((N, K), generator=g, device=DEV) * K ** -0.5)
    return data, scale, amax.view(-1)


def _rows_bf16(g, rows, K):
    x = torch.empty((rows, K), dtype=torch.bfloat16, device=DEV)
    for i in range(0, rows, 8192):
        n = min(8192, rows - i)
        x[i:i + n] = _rows_values(g, n, K).to(torch.bfloat16)
    return x


def _weights_i8(g, E, N, K):
    """8-bit weights of E experts, a scale for each of their N channels."""
    q = torch.empty((E, N, K), dtype=torch.int8, device=DEV)
    s = torch.empty((E, N), device=DEV)
    for e in range(E):
        w = torch.randn((N, K), generator=g, device=DEV) * K ** -0.5
        s[e] = w.abs().amax(1) / 127
        q[e] = torch.round(w / s[e][:, None]).to(torch.int8)
    return q, s


def _splits(seed, rows, E):
    """Skewed shares of the experts in groups of 128 rows; some are empty."""
    r = random.Random(int(seed) * 37 + 5)
    w = [(i + 1) ** -1.1 for i in range(E)]
    r.shuffle(w)
    if E > 4:
        w[r.randrange(E)] = 0.0
    units, tot = rows // ROW_GROUP, sum(w)
    share = [int(units * v / tot) for v in w]
    share[max(range(E), key=lambda i: w[i])] += units - sum(share)
    return [ROW_GROUP * v for v in share]


def _choices(g, T, E, k):
    """k different experts a token, some of them popular; the last token of a batch chooses none (padding)."""
    pop = torch.randn(E, generator=g, device=DEV) * 0.7
    ids = torch.topk(torch.randn((T, E), generator=g, device=DEV) + pop, k, dim=1).indices.to(torch.int32)
    if T > 8:
        ids[T - 1] = -1
    return ids.contiguous()


def _ends(seed, T, S):
    """Row ends of S sequences: uneven, some empty; a few rows may follow the last one."""
    r = random.Random(int(seed) * 41 + 3)
    last = T - (T // 50 if S > 1 else 0)
    cuts = sorted(r.randint(0, last) for _ in range(S - 1)) + [last]
    return torch.tensor(cuts, dtype=torch.int32, device=DEV)


def prepare(case, seed):
    c, op = dict(case), case["op"]
    g = _seeded(seed, 1)
    s = {"c": c}
    if op == "balance":
        T, E, k, S = c["T"], c["E"], c["k"], c["S"]
        l = torch.randn((T, E), generator=g, device=DEV) * 1.5 + 0.5 * torch.randn(E, generator=g, device=DEV)
        if T > 8:
            l[T - 1] = -float("inf")                               # a padding token
            l[T // 2, : E // 2] = -float("inf")                    # experts closed to a token
        s["logits"] = l.to(torch.bfloat16 if c["dtype"] == "bf16" else torch.float32)
        top = torch.topk(s["logits"].float(), k, dim=1)
        s["ids"] = torch.where(top.values > -float("inf"), top.indices, -1).to(torch.int32).contiguous()
        s["ends"] = _ends(seed, T, S) if S > 1 else None
        s["coef"] = 0.01
        s["dloss"] = 0.5 + torch.rand(1, generator=g, device=DEV)
        s["add"] = None
        if c["add"]:                                               # the gradient that came through the weights
            s["add"] = (torch.randn((T, E), generator=g, device=DEV) * (0.01 / T)).to(s["logits"].dtype)
        s.update(loss=torch.empty(1, device=DEV), counts=torch.empty((S, E), dtype=torch.int32, device=DEV),
                 probs=torch.empty((S, E), device=DEV), tokens=torch.empty(S, dtype=torch.int32, device=DEV),
                 dlogits=torch.empty_like(s["logits"]), workspace=torch.empty(1 << 23, dtype=torch.uint8, device=DEV))
    elif op == "keep8":
        M, E, H, F = c["M"], c["E"], c["H"], c["F"]
        s["splits"] = _splits(seed, M, E)
        s["a"], s["b"] = _rows_nvfp4(g, M, H), _weights_nvfp4(g, E, 2 * F, H)
        s["da"], s["db"] = _rows_nvfp4(g, M, H), _weights_nvfp4(g, E, F, H)
        b16 = dict(dtype=torch.bfloat16, device=DEV)
        s.update(h=torch.empty((M, F), **b16), again=torch.empty((M, F), **b16), dgu=torch.empty((M, 2 * F), **b16),
                 gu8=torch.empty((M, 2 * F), dtype=torch.int8, device=DEV),
                 gu_scale=torch.empty((2 * -(-F // KEEP_GROUP), M), **b16))
    elif op == "linear":
        T, N, K = c["T"], c["N"], c["K"]
        s["x"] = _rows_bf16(g, T, K)
        q, sc = _weights_i8(g, 1, N, K)
        s["b"] = (q[0], sc[0])
        s.update(q=torch.empty((T, K), dtype=torch.int8, device=DEV), scale=torch.empty(T, device=DEV),
                 out=torch.empty((T, N), dtype=torch.bfloat16 if c["out"] == "bf16" else torch.float32, device=DEV),
                 workspace=torch.empty(1 << 25, dtype=torch.uint8, device=DEV))
    elif op in ("experts", "experts_glu"):
        M, E = c["M"], c["E"]
        glu = op == "experts_glu"
        K, N = (c["H"], 2 * c["F"]) if glu else (c["K"], c["N"])
        cap = M + c.get("spare", 0)
        s["splits"] = _splits(seed, M, E)
        s["offs"] = torch.tensor(np.cumsum(s["splits"]), device=DEV).to(torch.int32)
        s["status"] = torch.zeros(1, dtype=torch.int32, device=DEV)
        s["x"] = _rows_bf16(g, cap, K)
        s["b"] = _weights_i8(g, E, N, K)
        s.update(q=torch.empty((cap, K), dtype=torch.int8, device=DEV), scale=torch.empty(cap, device=DEV))
        if glu:
            s["out"] = torch.empty((cap, c["F"]), dtype=torch.bfloat16, device=DEV)
        else:                                                      # rows past the last group stay as they are
            s["out"] = torch.zeros((cap, N), dtype=torch.bfloat16 if c["out"] == "bf16" else torch.float32, device=DEV)
    else:
        T, E, k, H, F = c["T"], c["E"], c["k"], c["H"], c["F"]
        s["ids"] = _choices(g, T, E, k)
        if op == "token_glu":
            s["x"] = _rows_bf16(g, T, H)
            s["b"] = _weights_i8(g, E, 2 * F, H)
            s["out"] = torch.empty((T * k, F), dtype=torch.bfloat16, device=DEV)
        else:
            s["x"] = _rows_bf16(g, T * k, F)
            s["b"] = _weights_i8(g, E, H, F)
            s["out"] = torch.empty((T * k, H), device=DEV)
    return s


# -------------------------------------------------------------- plain forms

def _decode(data, scale, amax):
    """f32 values of NVFP4 lines [..., L, K/2]."""
    lut = torch.tensor([v * sgn for sgn in (1.0, -1.0) for v in E2M1], device=data.device)
    both = torch.stack([lut.repeat(16), lut.repeat_interleave(16)], 1)
    v = both[data.int()].view(*scale.shape, 16)
    v = v * scale.view(torch.float8_e4m3fn).float()[..., None]
    return v.view(*scale.shape[:-1], -1) * (amax.view(scale.shape[:-1]) / 2688.0)[..., None]


def _act(g, kind):
    """The activation and its derivative."""
    if kind == "silu":
        q = 1 / (1 + torch.exp(-g))
        return g * q, q * (1 + g * (1 - q))
    u = 0.7978845608028654 * (g + 0.044715 * g * g * g)
    t = 1 - 2 / (1 + torch.exp(2 * u))
    return 0.5 * g * (1 + t), 0.5 * (1 + t) + 0.5 * g * (1 - t * t) * 0.7978845608028654 * (1 + 0.134145 * g * g)


def _segments(ends, T, S):
    """Sequence of each row (S for rows past the last) as an index."""
    t = torch.arange(T, device=DEV)
    return torch.zeros_like(t) if ends is None else torch.searchsorted(ends.long(), t, right=True)


def _balance(s):
    c = s["c"]
    T, E, k, S = c["T"], c["E"], c["k"], c["S"]
    l = s["logits"].float()
    on = l > -float("inf")
    at = _segments(s["ends"], T, S)
    if c["score"] == "sigmoid":
        sg = torch.where(on, 1 / (1 + torch.exp(-l)), torch.zeros_like(l))
        slope = 1 - sg
    else:
        sg = torch.where(on, torch.exp(l - l.amax(1, keepdim=True).clamp(min=-FLT_MAX)), torch.zeros_like(l))
        slope = 1
    p = sg / sg.sum(1, keepdim=True).clamp(min=1e-38)
    of = (at[None, :] == torch.arange(S, device=DEV)[:, None]).double()           # [S, T]: rows of each sequence
    probs = of @ p.double()
    tokens = (of @ on.any(1).double()[:, None]).view(S)
    chosen = torch.zeros((T, E + 1), device=DEV)                                    # whole numbers: 32 bits hold them
    chosen.scatter_add_(1, torch.where(s["ids"] >= 0, s["ids"], E).long(), torch.ones((T, k), device=DEV))
    counts = (of.float() @ chosen[:, :E]).double()
    n = tokens.double().clamp(min=1)
    w = s["coef"] * E / (k * S) / (n * n)
    loss = (w[:, None] * counts * probs).sum().view(1)
    a = torch.cat([w[:, None] * counts, torch.zeros((1, E), dtype=torch.float64, device=DEV)]).float() * s["dloss"]
    a = a[at]
    d = p * slope * (a - (p * a).sum(1, keepdim=True))
    if s["add"] is not None:
        d = d + s["add"].float()
    return {"loss": loss.float(), "counts": counts.int(), "probs": probs.float(), "tokens": tokens.int(),
            "dlogits": d.to(s["logits"].dtype)}


def _grouped(a, b, splits):
    """f32 [M, lines]: each expert's NVFP4 rows times its weight lines."""
    (ad, asc, aa), (bd, bsc, ba), ends = a, b, np.cumsum([0] + splits)
    ba = ba.view(len(splits), -1)
    return torch.cat([_decode(ad[i:j], asc[i:j], aa[i:j]) @ _decode(bd[e], bsc[e], ba[e]).t()
                      for e, (i, j) in enumerate(zip(ends[:-1], ends[1:])) if j > i])


def _kept(v):
    """The values that v [M, F] is kept as: 8-bit codes and a bf16 scale for 32 columns of a row."""
    M, F = v.shape
    pad = -F % KEEP_GROUP
    b = torch.cat([v, torch.zeros((M, pad), device=v.device)], 1).view(M, -1, KEEP_GROUP)
    sc = (b.abs().amax(2) / torch.full((), 127.0, device=v.device)).to(torch.bfloat16).float()[..., None]
    q = torch.where(sc > 0, torch.round(b / sc.clamp(min=1e-38)), torch.zeros_like(b)).clamp(-127, 127)
    return (q * sc).view(M, -1)[:, :F]


def _keep8(s):
    c = s["c"]
    g, u = _grouped(s["a"], s["b"], s["splits"]).chunk(2, 1)
    h = _act(g, c["act"])[0] * u
    g, u = _kept(g), _kept(u)
    dh = _grouped(s["da"], s["db"], s["splits"])
    a, da = _act(g, c["act"])
    return {"h": h.to(torch.bfloat16), "again": (a * u).to(torch.bfloat16),
            "dgu": torch.cat([dh * u * da, dh * a], 1).to(torch.bfloat16)}


def _cast_i8(x):
    """f32 codes [M, K] and f32 scales [M, 1] of rows."""
    x = x.float()
    amax = x.abs().amax(1, keepdim=True)
    top = torch.full_like(amax, 127.0)
    q = torch.round(x * torch.where(amax > 0, top / amax.clamp(min=1e-30), torch.zeros_like(amax)))
    return q, amax / top


def _tokens(s):
    """f32 [T*k, lines]: each choice's row in 8 bits times its expert's channels (zero where there is no choice)."""
    (bq, bs), c = s["b"], s["c"]
    q, sx = _cast_i8(s["x"])
    ids = s["ids"].reshape(-1)
    if q.shape[0] != ids.numel():
        q, sx = q.repeat_interleave(c["k"], 0), sx.repeat_interleave(c["k"], 0)
    used, back = torch.unique(ids.clamp(min=0), return_inverse=True)
    out = torch.zeros((q.shape[0], bq.shape[1]), device=q.device)
    for i, e in enumerate(used.tolist()):                          # the weights of one chosen expert at a time
        at = (back == i).nonzero().view(-1)
        out[at] = (q[at] @ bq[e].float().t()) * sx[at] * bs[e]
    return torch.where((ids >= 0)[:, None], out, torch.zeros_like(out))


def _experts(s):
    (bq, bs), ends = s["b"], np.cumsum([0] + s["splits"])
    q, sx = _cast_i8(s["x"][: int(ends[-1])])
    return torch.cat([(q[i:j] @ bq[e].float().t()) * sx[i:j] * bs[e]
                      for e, (i, j) in enumerate(zip(ends[:-1], ends[1:])) if j > i])


def _plain(s):
    c, op = s["c"], s["c"]["op"]
    if op == "balance":
        return _balance(s)
    if op == "keep8":
        return _keep8(s)
    if op == "linear":
        q, sx = _cast_i8(s["x"])
        return ((q @ s["b"][0].float().t()) * sx * s["b"][1]).to(s["out"].dtype)
    if op == "experts":
        out = _experts(s)
        more = s["out"].shape[0] - out.shape[0]
        return torch.cat([out, torch.zeros((more, out.shape[1]), device=out.device)]).to(s["out"].dtype)
    if op == "experts_glu":
        g, u = _experts(s).chunk(2, 1)
        return (_act(g, c["act"])[0] * u).to(torch.bfloat16)
    if op == "token_glu":
        g, u = _tokens(s).chunk(2, 1)
        return (_act(g, c["act"])[0] * u).to(torch.bfloat16)
    return _tokens(s)


# --------------------------------------------------------------- the kernels

def _kernels(s):
    from nvfp4_block_scaled_group_amd import i8, moe

    c, op = s["c"], s["c"]["op"]
    act = {"silu": moe.ACT_SILU, "gelu": moe.ACT_GELU}.get(c.get("act"))
    if op == "balance":
        how = dict(seq_ends=s["ends"], coef=s["coef"],
                   score=moe.SCORE_SOFTMAX if c["score"] == "softmax" else moe.SCORE_SIGMOID)
        moe.moe_balance(s["logits"], s["ids"], s["loss"], s["counts"], s["probs"], s["tokens"], s["workspace"], **how)
        moe.moe_balance_bwd(s["logits"], s["counts"], s["tokens"], s["dlogits"], topk=c["k"], dloss=s["dloss"],
                            add=s["add"], **how)
        return {key: s[key] for key in ("loss", "counts", "probs", "tokens", "dlogits")}
    if op == "keep8":
        moe.moe_glu_keep8(*s["a"], *s["b"], s["splits"], s["h"], s["gu8"], s["gu_scale"], act=act)
        moe.moe_glu_bwd_keep8(*s["da"], *s["db"], s["splits"], s["gu8"], s["gu_scale"], s["dgu"], h=s["again"], act=act)
        return {key: s[key] for key in ("h", "again", "dgu")}
    if op == "linear":
        i8.i8_group_cast(s["x"], s["q"], s["scale"])
        i8.i8_linear(s["q"], s["scale"], *s["b"], s["out"], s["workspace"])
        return s["out"]
    if op == "experts":
        i8.i8_group_cast_graphsafe(s["x"], s["offs"], s["q"], s["scale"], s["status"])
        i8.i8_group_gemm_graphsafe(s["q"], s["scale"], *s["b"], s["offs"], s["out"], s["status"])
        return s["out"]
    if op == "experts_glu":
        i8.i8_group_cast(s["x"], s["q"], s["scale"])
        i8.i8_group_glu(s["q"], s["scale"], *s["b"], s["splits"], s["out"], act=act)
        return s["out"]
    if op == "token_glu":
        i8.i8_token_glu(s["x"], s["ids"], *s["b"], s["out"], act=act)
        return s["out"]
    i8.i8_token_linear(s["x"], s["ids"], *s["b"], s["out"])
    return s["out"]


def run(state):
    return _kernels(state) if own else _plain(state)


# ---------------------------------------------------------------------- work

def work(case):
    c, op = case, case["op"]
    if op == "balance":
        T, E, k, S = c["T"], c["E"], c["k"], c["S"]
        n = 4 if c["dtype"] == "f32" else 2
        # the logits are needed again once the counts of a sequence are known
        return {"bytes": T * E * n * (4 if c["add"] else 3) + 4 * T * k + 12 * S * E, "flops": 16 * T * E}
    if op == "keep8":
        M, E, H, F = c["M"], c["E"], c["H"], c["F"]
        fixed = 0.5625 * H * (2 * M + E * 3 * F) + 4 * (2 * M + E * 3 * F)
        # h, h again, dgu; the kept values written and read once
        return {"bytes": fixed + 8 * M * F + 4 * M * F * (1 + 2 / KEEP_GROUP), "flops": 6.0 * M * H * F}
    if op == "linear":
        T, N, K = c["T"], c["N"], c["K"]
        return {"bytes": 2 * T * K + N * (K + 4) + T * N * (2 if c["out"] == "bf16" else 4), "flops": 2.0 * T * N * K}
    if op == "experts":
        M, E, N, K = c["M"], c["E"], c["N"], c["K"]
        return {"bytes": 2 * M * K + E * N * (K + 4) + M * N * (2 if c["out"] == "bf16" else 4), "flops": 2.0 * M * N * K}
    if op == "experts_glu":
        M, E, H, F = c["M"], c["E"], c["H"], c["F"]
        return {"bytes": 2 * M * H + E * 2 * F * (H + 4) + 2 * M * F, "flops": 4.0 * M * H * F}
    T, E, k, H, F = c["T"], c["E"], c["k"], c["H"], c["F"]
    t = T - 1 if T > 8 else T
    met = E * (1 - (1 - k / E) ** t)                               # experts that are chosen at all
    n, K = (2 * F, H) if op == "token_glu" else (H, F)
    moved = 2 * T * H + 2 * T * k * F if op == "token_glu" else 2 * T * k * F + 4 * T * k * H
    return {"bytes": met * n * (K + 4) + moved, "flops": 2.0 * t * k * n * K}


# --------------------------------------------------------------------- exact

def _lines64(data, scale, amax):
    """The values that NVFP4 lines stand for, by the formats' definitions, in 64 bits."""
    def e2m1(c):
        c = c.long()
        e, m = (c >> 1) & 3, (c & 1).double()
        v = torch.where(e == 0, 0.5 * m, torch.ldexp(1 + 0.5 * m, e - 1))
        return torch.where(c >= 8, -v, v)
    b = scale.long()
    e, m = b >> 3, (b & 7).double()
    S = torch.where(e == 0, m / 512, torch.ldexp(1 + m / 8, e - 7))
    v = torch.empty((*data.shape, 2), dtype=torch.float64, device=data.device)
    v[..., 0], v[..., 1] = e2m1(data & 15), e2m1(data >> 4)
    return v.view(*data.shape[:-1], -1) * S.repeat_interleave(16, -1) * (amax.double() / 2688)[..., None]


def _product64(a, b, splits):
    out, at = [], 0
    (ad, asc, aa), (bd, bsc, ba) = a, b
    lines = bd.shape[1]
    for e, m in enumerate(splits):
        w = _lines64(bd[e], bsc[e], ba[e * lines:(e + 1) * lines])
        for i in range(at, at + m, 4096):
            j = min(i + 4096, at + m)
            out.append(_lines64(ad[i:j], asc[i:j], aa[i:j]) @ w.T)
        at += m
    return torch.cat(out)


def _phi64(g, kind):
    if kind == "silu":
        q = torch.sigmoid(g)
        return g * q, q + g * q * (1 - q)
    c = (2 / np.pi) ** 0.5
    t = torch.tanh(c * (g + 0.044715 * g ** 3))
    return g * (1 + t) / 2, (1 + t) / 2 + g / 2 * (1 - t ** 2) * c * (1 + 3 * 0.044715 * g ** 2)


def _kept64(v):
    """In place: each group of columns becomes the multiples of its scale that are nearest."""
    for i in range(0, v.shape[1], KEEP_GROUP):
        w = v[:, i:i + KEEP_GROUP]
        step = (w.abs().max(1, keepdim=True).values / 127).to(torch.bfloat16).double()
        v[:, i:i + KEEP_GROUP] = torch.where(step > 0, torch.round(w / step) * step, 0 * w)
    return v


def _codes64(x):
    """Codes and scales of rows by their definition: a code is the nearest whole number to the fp32 product of the
    value and 127 / amax (fp32); the scale is amax / 127."""
    amax = np.abs(x).max(1, keepdims=True).astype(np.float32)
    inv = np.divide(np.float32(127), amax, out=np.zeros_like(amax), where=amax > 0)
    return torch.from_numpy(np.rint(x.astype(np.float32) * inv).astype(np.float64)).to(DEV), \
        torch.from_numpy(amax.astype(np.float64) / 127).to(DEV)


def _i8_64(x, bq, bs):
    """Rows times channels in whole numbers (64 bits hold them exactly), then the scales."""
    out = []
    for i in range(0, x.shape[0], 8192):
        q, sx = _codes64(x[i:i + 8192].float().cpu().numpy())
        out.append((q @ bq.double().T) * sx * bs.double())
    return torch.cat(out)


def _balance64(s):
    c = s["c"]
    T, E, k, S = c["T"], c["E"], c["k"], c["S"]
    l = s["logits"].double().cpu().numpy()
    ids = s["ids"].cpu().numpy()
    ends = [T] if s["ends"] is None else s["ends"].tolist()
    grad = np.zeros((T, E)) if s["add"] is None else s["add"].double().cpu().numpy()
    loss, counts, probs, tokens, begin = 0.0, np.zeros((S, E)), np.zeros((S, E)), np.zeros(S), 0
    for j, end in enumerate(ends):
        z, chosen = l[begin:end], ids[begin:end].reshape(-1)
        open_ = np.isfinite(z)
        counts[j] = np.bincount(chosen[chosen >= 0], minlength=E)
        tokens[j] = n = int(open_.any(1).sum())
        if n:
            with np.errstate(all="ignore"):
                sg = np.where(open_, 1 / (1 + np.exp(-z)) if c["score"] == "sigmoid" else np.exp(z - z.max(1, keepdims=True)), 0)
                p = np.where(open_.any(1, keepdims=True), sg / sg.sum(1, keepdims=True), 0)
            probs[j] = p.sum(0)
            a = s["coef"] / S * E / k * counts[j] / n / n
            loss += float(a @ probs[j])
            d = p * (a - p @ a[:, None])
            if c["score"] == "sigmoid":
                d = d * (1 - sg)
            grad[begin:end] += float(s["dloss"]) * d
        begin = end
    return {"loss": torch.tensor([loss], dtype=torch.float64), "counts": None, "probs": torch.from_numpy(probs), "tokens": None,
            "dlogits": torch.from_numpy(grad)}


def exact(case, seed):
    s = prepare(case, seed)
    c, op = s["c"], s["c"]["op"]
    if op == "balance":
        return _balance64(s)
    if op == "keep8":
        F = c["F"]
        gu = _product64(s["a"], s["b"], s["splits"])
        h = _phi64(gu[:, :F], c["act"])[0] * gu[:, F:]
        g, u = _kept64(gu[:, :F].clone()), _kept64(gu[:, F:].clone())
        del gu
        dh = _product64(s["da"], s["db"], s["splits"])
        a, da = _phi64(g, c["act"])
        return {"h": h, "again": a * u, "dgu": torch.cat([dh * u * da, dh * a], 1)}
    bq, bs = s["b"]
    if op == "linear":
        return _i8_64(s["x"], bq, bs)
    if op in ("experts", "experts_glu"):
        out, at = torch.zeros((s["x"].shape[0], bq.shape[1]), dtype=torch.float64, device=DEV), 0
        for e, m in enumerate(s["splits"]):
            if m:
                out[at:at + m] = _i8_64(s["x"][at:at + m], bq[e], bs[e])
            at += m
        if op == "experts":
            return out
        return _phi64(out[:, : c["F"]], c["act"])[0] * out[:, c["F"]:]
    ids, k = s["ids"].cpu().numpy(), c["k"]
    out = torch.zeros((ids.size, bq.shape[1]), dtype=torch.float64, device=DEV)
    for e in range(c["E"]):
        t, j = np.nonzero(ids == e)
        if t.size:
            p = torch.from_numpy(t * k + j).to(DEV)
            out[p] = _i8_64(s["x"][p if op == "token_down" else torch.from_numpy(t).to(DEV)], bq[e], bs[e])
    if op == "token_down":
        return out
    return _phi64(out[:, : c["F"]], c["act"])[0] * out[:, c["F"]:]

"""Cases of the mixture-of-experts and adapter operators, with their plain forms.

Three operators are listed here:

* routing: selection of experts with weights and the 128-row padded plan
  (``moe_route``, ``moe_plan``), the movement of rows into and out of that plan
  (``moe_dispatch``, ``moe_combine``) and the gradients of both;
* the gated feed-forward block of the experts on row-scaled NVFP4 operands
  (``moe_glu``, ``moe_glu_bwd``) and its form for single tokens
  (``moe_token_glu``, ``moe_token_linear``);
* low-rank adapters of many requests beside one shared NVFP4 projection
  (``lora_linear``).

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
FLT_MAX = 3.4028234663852886e38
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ------------------------------------------------------------------- cases

def listed():
    return [
        # one token of a decoding request: 256 experts, 8 chosen; latency counts
        dict(name="route_token", op="route", T=1, E=256, k=8, dtype="f32", score="softmax", norm=True, bias=False),
        # a large training batch, sigmoid scores with a balancing bias on the selection
        dict(name="route_batch", op="route", T=32768, E=256, k=8, dtype="f32", score="sigmoid", norm=True, bias=True),
        # gradient of the weights, bf16 logits, an odd number of tokens
        dict(name="route_grad", op="route_grad", T=8191, E=64, k=6, dtype="bf16", score="softmax", norm=False,
             bias=False),
        # a batch's tokens copied into the experts' packed rows (one device's share of 32 experts)
        dict(name="dispatch_batch", op="dispatch", T=8192, E=32, k=8, H=7168),
        # the experts' results of a few decoding requests brought back to their tokens
        dict(name="combine_tokens", op="combine", T=33, E=64, k=6, H=2064, y="bf16"),
        # gradient of the combine: rows and weights, fp32 results of the grouped GEMM
        dict(name="combine_grad", op="combine_grad", T=4095, E=64, k=6, H=2048, y="f32"),
        # gate and up projection of a batch, skewed routing over 32 experts
        dict(name="glu_batch", op="glu", M=65536, E=32, H=7168, F=2048, act="silu", keep=True),
        # backward through the down projection and the activation
        dict(name="glu_grad", op="glu_grad", M=16384, E=64, H=2048, F=1040, act="gelu"),
        # one decoding token: the 8 chosen experts' gate and up weights are read once
        dict(name="glu_token", op="glu_token", T=1, E=32, k=8, H=7168, F=2048, act="silu"),
        # a ragged decoding batch: several tokens meet in some experts; down projection
        dict(name="down_tokens", op="down_token", T=24, E=64, k=6, H=7168, F=2048),
        # eight requests, one token each, with six adapters
        dict(name="lora_tokens", op="lora", T=8, N=7168, K=7168, R=16, n=6, mix="tokens"),
        # prompts of several requests in one batch, each with its adapter
        dict(name="lora_prompts", op="lora", T=4095, N=7168, K=2048, R=32, n=8, mix="prompts"),
    ]


def _log(rng, lo, hi):
    """A whole number between lo and hi, spread over its logarithm."""
    v = int(round(lo * (hi / lo) ** rng.random()))
    return max(lo, min(hi, v))


def draw(rng):
    op = rng.choice(["route", "route_grad", "dispatch", "combine", "combine_grad", "glu", "glu_grad", "glu_token",
                     "down_token", "lora", "lora"])
    if op in ("route", "route_grad"):
        E = rng.choice([8, 16, 40, 64, 100, 128, 160, 256, 384, 512])
        T = _log(rng, 1, 32768 * 256 // E if E >= 256 else 32768)
        return dict(op=op, T=T, E=E, k=rng.randint(1, min(E, 10)), dtype=rng.choice(["f32", "bf16"]),
                    score=rng.choice(["softmax", "sigmoid"]), norm=rng.random() < 0.5, bias=rng.random() < 0.5)
    if op in ("dispatch", "combine", "combine_grad"):
        H = 16 * _log(rng, 16, 448)
        c = dict(op=op, T=_log(rng, 1, min(32768, 8192 * 7168 // H)), E=rng.choice([8, 32, 60, 64, 128]),
                 k=rng.randint(1, 8), H=H)
        if op != "dispatch":
            c["y"] = rng.choice(["f32", "bf16"])
        return c
    if op in ("glu", "glu_grad"):
        c = dict(op=op, M=ROW_GROUP * _log(rng, 1, 256), E=rng.choice([1, 4, 8, 16, 32, 64]),
                 H=128 * _log(rng, 2, 56), F=16 * _log(rng, 8, 128), act=rng.choice(["silu", "gelu"]))
        if op == "glu":
            c["keep"] = rng.random() < 0.5
        return c
    if op in ("glu_token", "down_token"):
        E = rng.choice([1, 8, 16, 32, 64])
        c = dict(op=op, T=_log(rng, 1, 64), E=E, k=rng.randint(1, min(E, 8)), H=32 * _log(rng, 8, 224),
                 F=32 * _log(rng, 8, 64))
        if op == "glu_token":
            c["act"] = rng.choice(["silu", "gelu"])
        return c
    return dict(op="lora", T=_log(rng, 1, 8192), N=16 * _log(rng, 16, 448), K=32 * _log(rng, 8, 224),
                R=8 * rng.randint(1, 8), n=rng.randint(1, 32), mix=rng.choice(["tokens", "prompts"]))


# ------------------------------------------------------------------- inputs

def _seeded(seed, salt):
    g = torch.Generator(device=DEV)
    g.manual_seed((int(seed) * 1000003 + salt * 7919 + 17) % (1 << 62))
    return g


def _cast_lines(x):
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


def _rows_nvfp4(g, rows, K):
    """Activation rows: normal values times a row scale, as packed MoE activations have them."""
    data = torch.empty((rows, K // 2), dtype=torch.uint8, device=DEV)
    scale = torch.empty((rows, K // 16), dtype=torch.uint8, device=DEV)
    amax = torch.empty(rows, device=DEV)
    for i in range(0, rows, 8192):
        n = min(8192, rows - i)
        x = torch.randn((n, K), generator=g, device=DEV) * torch.exp(0.5 * torch.randn((n, 1), generator=g, device=DEV))
        data[i:i + n], scale[i:i + n], amax[i:i + n] = _cast_lines(x)
    return data, scale, amax


def _weights_nvfp4(g, E, N, K):
    """Weights of E experts, N lines of K each, with the spread that keeps outputs near one."""
    data = torch.empty((E, N, K // 2), dtype=torch.uint8, device=DEV)
    scale = torch.empty((E, N, K // 16), dtype=torch.uint8, device=DEV)
    amax = torch.empty((E, N), device=DEV)
    for e in range(E):
        data[e], scale[e], amax[e] = _cast_lines(torch.randn((N, K), generator=g, device=DEV) * K ** -0.5)
    return data, scale, amax.view(-1)


def _bf16(g, *shape, scale=1.0):
    return (torch.randn(shape, generator=g, device=DEV) * scale).to(torch.bfloat16)


def _splits(seed, rows, E):
    """Skewed shares of the experts in groups of 128 rows; some are empty."""
    r = random.Random(int(seed) * 31 + 7)
    w = [(i + 1) ** -1.1 for i in range(E)]
    r.shuffle(w)
    if E > 4:
        w[r.randrange(E)] = 0.0
    units, tot = rows // ROW_GROUP, sum(w)
    share = [int(units * v / tot) for v in w]
    share[max(range(E), key=lambda i: w[i])] += units - sum(share)
    return [ROW_GROUP * v for v in share]


def _capacity(T, k, E):
    """Rows that T*k choices can take at most once every expert's group is padded."""
    n = T * k
    return min(n * ROW_GROUP, (n + E * (ROW_GROUP - 1)) // ROW_GROUP * ROW_GROUP)


def _choices(g, T, E, k):
    """k different experts a token, some of them popular; the last token of a batch chooses none (padding)."""
    pop = torch.randn(E, generator=g, device=DEV) * 0.7
    ids = torch.topk(torch.randn((T, E), generator=g, device=DEV) + pop, k, dim=1).indices.to(torch.int32)
    if T > 8:
        ids[T - 1] = -1
    return ids.contiguous()


def _plan_of(ids, E, cap):
    """rows [T, k], src [cap], ends [E], counts [E] of the choices, groups padded to 128 rows."""
    T, k = ids.shape
    flat = ids.reshape(-1).long()
    flat = torch.where((flat >= 0) & (flat < E), flat, torch.full_like(flat, E))
    order = torch.sort(flat, stable=True).indices
    counts = torch.bincount(flat, minlength=E + 1)[:E]
    padded = (counts + ROW_GROUP - 1) // ROW_GROUP * ROW_GROUP
    ends = torch.cumsum(padded, 0)
    first = torch.cumsum(counts, 0) - counts                      # an expert's first place in the sorted pairs
    shift = torch.cat([ends - padded - first, torch.zeros(1, dtype=torch.long, device=ids.device)])
    e = flat[order]
    row = torch.arange(T * k, device=ids.device) + shift[e]
    row = torch.where(e < E, row, torch.full_like(row, -1))
    rows = torch.empty(T * k, dtype=torch.int32, device=ids.device)
    rows[order] = row.to(torch.int32)
    src = torch.full((cap + 1,), -1, dtype=torch.int32, device=ids.device)
    src[torch.where(row >= 0, row, torch.full_like(row, cap))] = order.to(torch.int32)
    return rows.view(T, k), src[:cap].clone(), ends.to(torch.int32), counts.to(torch.int32)


def prepare(case, seed):
    c, op = dict(case), case["op"]
    g = _seeded(seed, 1)
    s = {"c": c}
    if op in ("route", "route_grad"):
        T, E, k = c["T"], c["E"], c["k"]
        l = torch.randn((T, E), generator=g, device=DEV) * 1.5
        if T > 8:
            l[T - 1] = -float("inf")                               # a padding token
            l[T // 2, : E // 2] = -float("inf")                    # experts closed to a token
        s["logits"] = l.to(torch.bfloat16 if c["dtype"] == "bf16" else torch.float32)
        s["bias"] = torch.randn(E, generator=g, device=DEV) * 0.1 if c["bias"] else None
        s["ids"] = torch.empty((T, k), dtype=torch.int32, device=DEV)
        s["weights"] = torch.empty((T, k), device=DEV)
        if op == "route":
            cap = _capacity(T, k, E)
            s.update(cap=cap, offs=torch.empty(E, dtype=torch.int32, device=DEV),
                     counts=torch.empty(E, dtype=torch.int32, device=DEV),
                     rows=torch.empty((T, k), dtype=torch.int32, device=DEV),
                     src=torch.empty(cap, dtype=torch.int32, device=DEV),
                     status=torch.zeros(1, dtype=torch.int32, device=DEV))
            s["workspace"] = torch.empty(1 << 23, dtype=torch.uint8, device=DEV)
        else:
            s["ids"], _ = _select(s["logits"], s["bias"], c)
            s["dweights"] = torch.randn((T, k), generator=g, device=DEV)
            s["dlogits"] = torch.empty_like(s["logits"])
    elif op in ("dispatch", "combine", "combine_grad"):
        T, E, k, H = c["T"], c["E"], c["k"], c["H"]
        cap = _capacity(T, k, E)
        s["rows"], s["src"], s["offs"], _ = _plan_of(_choices(g, T, E, k), E, cap)
        s["cap"] = cap
        if op != "combine":
            s["x"] = _bf16(g, T, H)
            s["out"] = torch.zeros((cap, H), dtype=torch.bfloat16, device=DEV)
        if op != "dispatch":
            w = torch.rand((T, k), generator=g, device=DEV)
            s["w"] = w / w.sum(1, keepdim=True)
            y = torch.randn((cap, H), generator=g, device=DEV)
            s["y"] = y.to(torch.bfloat16) if c["y"] == "bf16" else y
        if op == "combine":
            s["out"] = torch.empty((T, H), dtype=torch.bfloat16, device=DEV)
        if op == "combine_grad":
            s["dw"] = torch.empty((T, k), device=DEV)
    elif op in ("glu", "glu_grad"):
        M, E, H, F = c["M"], c["E"], c["H"], c["F"]
        s["splits"] = _splits(seed, M, E)
        s["a"] = _rows_nvfp4(g, M, H)
        s["b"] = _weights_nvfp4(g, E, 2 * F if op == "glu" else F, H)
        if op == "glu":
            s["h"] = torch.empty((M, F), dtype=torch.bfloat16, device=DEV)
            s["gu"] = torch.empty((M, 2 * F), dtype=torch.bfloat16, device=DEV) if c["keep"] else None
        else:
            s["gu"] = _bf16(g, M, 2 * F)
            s["dgu"] = torch.empty((M, 2 * F), dtype=torch.bfloat16, device=DEV)
    elif op in ("glu_token", "down_token"):
        T, E, k, H, F = c["T"], c["E"], c["k"], c["H"], c["F"]
        s["ids"] = _choices(g, T, E, k)
        if op == "glu_token":
            s["x"] = _bf16(g, T, H)
            s["b"] = _weights_nvfp4(g, E, 2 * F, H)
            s["out"] = torch.empty((T * k, F), dtype=torch.bfloat16, device=DEV)
        else:
            s["x"] = _bf16(g, T * k, F)
            s["b"] = _weights_nvfp4(g, E, H, F)
            s["out"] = torch.empty((T * k, H), device=DEV)
    else:
        T, N, K, R, n = c["T"], c["N"], c["K"], c["R"], c["n"]
        s["x"] = _bf16(g, T, K)
        s["b"] = _weights_nvfp4(g, 1, N, K)
        s["A"] = _bf16(g, n, R, K, scale=K ** -0.5)
        s["B"] = _bf16(g, n, N, R, scale=R ** -0.5)
        s["cs"] = 0.5 + torch.rand(n, generator=g, device=DEV)
        if c["mix"] == "tokens":                                   # every row a request of its own
            a = torch.randint(-1, n, (T,), generator=g, device=DEV)
        else:                                                      # runs of rows, one request each
            cuts = torch.rand((T,), generator=g, device=DEV) < max(1.0 / max(T, 1), 0.004)
            a = (torch.cumsum(cuts.long(), 0) * 7 + int(seed)) % (n + 1) - 1
        s["aid"] = a.to(torch.int32)
        s["out"] = torch.empty((T, N), dtype=torch.bfloat16, device=DEV)
        s["workspace"] = torch.empty(1 << 25, dtype=torch.uint8, device=DEV)
    return s


# -------------------------------------------------------------- plain forms

def _decode(data, scale, amax):
    """f32 values of NVFP4 lines [..., L, K/2]."""
    lut = torch.tensor([v * sgn for sgn in (1.0, -1.0) for v in E2M1], device=data.device)
    both = torch.stack([lut.repeat(16), lut.repeat_interleave(16)], 1)
    v = both[data.int()].view(*scale.shape, 16)
    v = v * scale.view(torch.float8_e4m3fn).float()[..., None]
    return v.view(*scale.shape[:-1], -1) * (amax.view(scale.shape[:-1]) / 2688.0)[..., None]


def _select(logits, bias, c):
    """ids [T, k] (ties to the lower index, -1 for no expert) and the unmasked logits, f32."""
    l = logits.float()
    l = torch.where(l > -float("inf"), l.clamp(max=FLT_MAX), torch.full_like(l, -float("inf")))
    key = l + bias if bias is not None else l
    top, at = torch.sort(key, dim=1, descending=True, stable=True)
    at = at[:, : c["k"]].to(torch.int32)
    return torch.where(top[:, : c["k"]] > -float("inf"), at, torch.full_like(at, -1)).contiguous(), l


def _scores(l, ids, c):
    """Chosen logits, whether each choice is one, and the chosen scores before scaling (unnormalised)."""
    on = ids >= 0
    chosen = torch.where(on, torch.gather(l, 1, ids.clamp(min=0).long()), torch.full_like(ids, -float("inf"), dtype=l.dtype))
    if c["score"] == "sigmoid":
        return chosen, on, torch.where(on, 1 / (1 + torch.exp(-chosen)), torch.zeros_like(chosen))
    over = chosen if c["norm"] else l
    top = over.amax(1, keepdim=True).clamp(min=-FLT_MAX)
    return chosen, on, torch.exp(chosen - top) / torch.exp(over - top).sum(1, keepdim=True).clamp(min=1e-38)


def _route(s):
    c = s["c"]
    ids, l = _select(s["logits"], s["bias"], c)
    _, _, p = _scores(l, ids, c)
    if c["norm"] and c["score"] == "sigmoid":
        tot = p.sum(1, keepdim=True)
        p = torch.where(tot > 0, p / tot.clamp(min=1e-38), torch.zeros_like(p))
    rows, src, ends, counts = _plan_of(ids, c["E"], s["cap"])
    return {"ids": ids, "weights": p * 2.5, "rows": rows, "src": src, "offs": ends, "counts": counts}


def _route_grad(s):
    c = s["c"]
    ids, l = s["ids"], s["logits"].float()
    chosen, on, p = _scores(l, ids, c)
    g = torch.where(on, s["dweights"] * 2.5, torch.zeros_like(p))
    at = ids.clamp(min=0).long()
    dl = torch.zeros_like(l)
    if c["score"] == "sigmoid" and c["norm"]:
        q = p / p.sum(1, keepdim=True).clamp(min=1e-38)
        d = (g - (q * g).sum(1, keepdim=True)) * q * (1 - p)
    elif c["score"] == "sigmoid":
        d = g * p * (1 - p)
    else:
        inner = (p * g).sum(1, keepdim=True)
        d = p * g if not c["norm"] else p * (g - inner)
        if not c["norm"]:
            top = l.amax(1, keepdim=True).clamp(min=-FLT_MAX)
            e = torch.exp(l - top)
            dl = -inner * e / e.sum(1, keepdim=True).clamp(min=1e-38)
    dl = dl.scatter_add(1, at, torch.where(on, d, torch.zeros_like(d)))
    return dl.to(s["logits"].dtype)


def _act(g, kind):
    """The activation and its derivative."""
    if kind == "silu":
        q = 1 / (1 + torch.exp(-g))
        return g * q, q * (1 + g * (1 - q))
    u = 0.7978845608028654 * (g + 0.044715 * g * g * g)
    t = 1 - 2 / (1 + torch.exp(2 * u))
    return 0.5 * g * (1 + t), 0.5 * (1 + t) + 0.5 * g * (1 - t * t) * 0.7978845608028654 * (1 + 0.134145 * g * g)


def _grouped(s):
    """f32 [M, lines]: each expert's rows times its weight lines."""
    (ad, asc, aa), (bd, bsc, ba), E = s["a"], s["b"], s["c"]["E"]
    ba, ends = ba.view(E, -1), np.cumsum([0] + s["splits"])
    return torch.cat([_decode(ad[i:j], asc[i:j], aa[i:j]) @ _decode(bd[e], bsc[e], ba[e]).t()
                      for e, (i, j) in enumerate(zip(ends[:-1], ends[1:])) if j > i])


def _tokens(s):
    """f32 [T*k, lines]: each choice's row times its expert's weight lines (zero where there is no choice)."""
    (bd, bsc, ba), c = s["b"], s["c"]
    ids, x = s["ids"].reshape(-1), s["x"].float()
    if x.shape[0] != ids.numel():
        x = x.repeat_interleave(c["k"], 0)
    used, back = torch.unique(ids.clamp(min=0), return_inverse=True)
    ba = ba.view(c["E"], -1)
    out = torch.zeros((x.shape[0], bd.shape[1]), device=x.device)
    for i, e in enumerate(used.tolist()):                          # the weights of one chosen expert at a time
        at = (back == i).nonzero().view(-1)
        out[at] = x[at] @ _decode(bd[e], bsc[e], ba[e]).t()
    return torch.where((ids >= 0)[:, None], out, torch.zeros_like(out))


def _lora(s):
    x, aid = s["x"].float(), s["aid"].long()
    y = x @ _decode(s["b"][0][0], s["b"][1][0], s["b"][2]).t()
    n, R, K = s["A"].shape
    # every row times every adapter's A, the other adapters' columns masked out: one product each way
    v = (x @ s["A"].float().view(n * R, K).t()).view(-1, n, R)
    mine = torch.arange(n, device=x.device)[None, :] == aid[:, None]
    v = torch.where(mine[..., None], v * s["cs"][None, :, None], torch.zeros_like(v)).view(-1, n * R)
    return (y + v @ s["B"].float().transpose(0, 1).reshape(-1, n * R).t()).to(torch.bfloat16)


def _plain(s):
    c, op = s["c"], s["c"]["op"]
    if op == "route":
        return _route(s)
    if op == "route_grad":
        return _route_grad(s)
    if op == "dispatch":
        row = s["src"] >= 0
        x = s["x"].float()[s["src"].clamp(min=0).long() // c["k"]]
        return torch.where(row[:, None], x, torch.zeros_like(x)).to(torch.bfloat16)
    if op == "combine":
        on, at = s["rows"] >= 0, s["rows"].clamp(min=0).long()
        return (s["y"][at].float() * torch.where(on, s["w"], torch.zeros_like(s["w"]))[..., None]).sum(1).to(torch.bfloat16)
    if op == "combine_grad":
        on, at, row = s["rows"] >= 0, s["rows"].clamp(min=0).long(), s["src"] >= 0
        x, pair = s["x"].float(), s["src"].clamp(min=0).long()
        dy = x[pair // c["k"]] * torch.where(row, s["w"].view(-1)[pair], torch.zeros_like(pair, dtype=torch.float32))[:, None]
        dw = (s["y"][at].float() * x[:, None, :]).sum(2)
        return {"dy": dy.to(torch.bfloat16), "dw": torch.where(on, dw, torch.zeros_like(dw))}
    if op == "glu":
        gu = _grouped(s)
        g, u = gu.chunk(2, 1)
        return {"h": (_act(g, c["act"])[0] * u).to(torch.bfloat16), "gu": gu.to(torch.bfloat16) if c["keep"] else None}
    if op == "glu_grad":
        dh = _grouped(s)
        g, u = s["gu"].float().chunk(2, 1)
        a, da = _act(g, c["act"])
        return torch.cat([dh * u * da, dh * a], 1).to(torch.bfloat16)
    if op == "glu_token":
        g, u = _tokens(s).chunk(2, 1)
        return (_act(g, c["act"])[0] * u).to(torch.bfloat16)
    return _tokens(s) if op == "down_token" else _lora(s)


# --------------------------------------------------------------- the kernels

def _kernels(s):
    from nvfp4_block_scaled_group_amd import moe

    c, op = s["c"], s["c"]["op"]
    score = {"softmax": moe.SCORE_SOFTMAX, "sigmoid": moe.SCORE_SIGMOID}.get(c.get("score"))
    act = {"silu": moe.ACT_SILU, "gelu": moe.ACT_GELU}.get(c.get("act"))
    if op == "route":
        moe.moe_route(s["logits"], s["ids"], s["weights"], select_bias=s["bias"], score=score, normalize=c["norm"], scale=2.5)
        moe.moe_plan(s["ids"], s["offs"], s["counts"], s["rows"], s["src"], s["status"], s["workspace"])
        return {key: s[key] for key in ("ids", "weights", "rows", "src", "offs", "counts")}
    if op == "route_grad":
        moe.moe_route_bwd(s["logits"], s["ids"], s["dweights"], s["dlogits"], score=score, normalize=c["norm"], scale=2.5)
        return s["dlogits"]
    if op == "dispatch":
        moe.moe_dispatch(s["x"], s["rows"], s["src"], s["offs"], s["out"])
        return s["out"]
    if op == "combine":
        moe.moe_combine(s["y"], s["rows"], s["out"], weights=s["w"])
        return s["out"]
    if op == "combine_grad":
        moe.moe_dispatch(s["x"], s["rows"], s["src"], s["offs"], s["out"], weights=s["w"], y=s["y"], dweights=s["dw"])
        return {"dy": s["out"], "dw": s["dw"]}
    if op == "glu":
        moe.moe_glu(*s["a"], *s["b"], s["splits"], s["h"], gu=s["gu"], act=act)
        return {"h": s["h"], "gu": s["gu"]}
    if op == "glu_grad":
        moe.moe_glu_bwd(*s["a"], *s["b"], s["splits"], s["gu"], s["dgu"], act=act)
        return s["dgu"]
    if op == "glu_token":
        moe.moe_token_glu(s["x"], s["ids"], *s["b"], s["out"], act=act)
        return s["out"]
    if op == "down_token":
        moe.moe_token_linear(s["x"], s["ids"], *s["b"], s["out"])
        return s["out"]
    moe.lora_linear(s["x"], s["b"][0][0], s["b"][1][0], s["b"][2], s["A"], s["B"], s["aid"], s["cs"], s["out"], s["workspace"])
    return s["out"]


def run(state):
    return _kernels(state) if own else _plain(state)


# ---------------------------------------------------------------------- work

def work(case):
    c, op = case, case["op"]
    if op == "route":
        T, E, k = c["T"], c["E"], c["k"]
        return {"bytes": T * E * (4 if c["dtype"] == "f32" else 2) + 12 * T * k + 4 * _capacity(T, k, E) + 8 * E,
                "flops": 4 * T * E}
    if op == "route_grad":
        T, E, k = c["T"], c["E"], c["k"]
        return {"bytes": 2 * T * E * (4 if c["dtype"] == "f32" else 2) + 8 * T * k, "flops": 4 * T * E}
    if op in ("dispatch", "combine", "combine_grad"):
        T, k, H = c["T"], c["k"], c["H"]
        n = (T - 1 if T > 8 else T) * k                            # rows in use
        y = 4 if c.get("y") == "f32" else 2
        if op == "dispatch":
            return {"bytes": 2 * T * H + 2 * n * H + 8 * T * k, "flops": 0}
        if op == "combine":
            return {"bytes": 2 * T * H + y * n * H + 8 * T * k, "flops": 2 * n * H}
        return {"bytes": 2 * T * H + (2 + y) * n * H + 16 * T * k, "flops": 3 * n * H}
    if op in ("glu", "glu_grad"):
        M, E, H, F = c["M"], c["E"], c["H"], c["F"]
        n = 2 * F if op == "glu" else F
        fixed = 0.5625 * H * (M + E * n) + 4 * (M + E * n)
        moved = 2 * M * F + (4 * M * F if c.get("keep") else 0) if op == "glu" else 8 * M * F
        return {"bytes": fixed + moved, "flops": 2.0 * M * H * n}
    if op in ("glu_token", "down_token"):
        T, E, k, H, F = c["T"], c["E"], c["k"], c["H"], c["F"]
        t = T - 1 if T > 8 else T
        met = E * (1 - (1 - k / E) ** t)                           # experts that are chosen at all
        n, K = (2 * F, H) if op == "glu_token" else (H, F)
        moved = 2 * T * H + 2 * T * k * F if op == "glu_token" else 2 * T * k * F + 4 * T * k * H
        return {"bytes": met * n * (0.5625 * K + 4) + moved, "flops": 2.0 * t * k * n * K}
    T, N, K, R, n = c["T"], c["N"], c["K"], c["R"], c["n"]
    met = n * (1 - (1 - 1 / (n + 1)) ** (T if c["mix"] == "tokens" else max(1, T * 0.004)))
    return {"bytes": N * (0.5625 * K + 4) + met * 2 * R * (N + K) + 2 * T * (N + K),
            "flops": 2.0 * T * N * K + 2.0 * T * R * (N + K) * n / (n + 1)}


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
    lo, hi = e2m1(data & 15), e2m1(data >> 4)
    v = torch.empty((*data.shape, 2), dtype=torch.float64, device=data.device)
    v[..., 0], v[..., 1] = lo, hi
    return v.view(*data.shape[:-1], -1) * S.repeat_interleave(16, -1) * (amax.double() / 2688)[..., None]


def _phi64(g, kind):
    if kind == "silu":
        q = torch.sigmoid(g)
        return g * q, q + g * q * (1 - q)
    c = (2 / np.pi) ** 0.5
    t = torch.tanh(c * (g + 0.044715 * g ** 3))
    return g * (1 + t) / 2, (1 + t) / 2 + g / 2 * (1 - t ** 2) * c * (1 + 3 * 0.044715 * g ** 2)


def _product64(s):
    out, at = [], 0
    (ad, asc, aa), (bd, bsc, ba) = s["a"], s["b"]
    lines = bd.shape[1]
    for e, m in enumerate(s["splits"]):
        w = _lines64(bd[e], bsc[e], ba[e * lines:(e + 1) * lines])
        for i in range(at, at + m, 4096):
            j = min(i + 4096, at + m)
            out.append(_lines64(ad[i:j], asc[i:j], aa[i:j]) @ w.T)
        at += m
    return torch.cat(out)


def _pairs64(s):
    bd, bsc, ba = s["b"]
    lines, k = bd.shape[1], s["c"]["k"]
    ids, x = s["ids"].cpu().numpy(), s["x"].double()
    out = torch.zeros((ids.size, lines), dtype=torch.float64, device=x.device)
    for e in range(bd.shape[0]):
        t, j = np.nonzero(ids == e)
        if t.size:
            p = torch.from_numpy(t * k + j).to(x.device)
            rows = p if x.shape[0] == ids.size else torch.from_numpy(t).to(x.device)
            out[p] = x[rows] @ _lines64(bd[e], bsc[e], ba[e * lines:(e + 1) * lines]).T
    return out


def _weights64(s, ids):
    """Scaled weights and their gradient with respect to the logits, from numpy in 64 bits."""
    c = s["c"]
    l = s["logits"].double().cpu().numpy()
    T, k = ids.shape
    w, jac = np.zeros((T, k)), None
    dl = np.zeros_like(l)
    dw = s["dweights"].double().cpu().numpy() if "dweights" in s else np.zeros((T, k))
    t, j = np.nonzero(ids >= 0)
    z = np.full((T, k), -np.inf)
    z[t, j] = l[t, ids[t, j]]
    with np.errstate(all="ignore"):
        if c["score"] == "sigmoid":
            sg = np.where(ids >= 0, 1 / (1 + np.exp(-z)), 0.0)
            tot = sg.sum(1, keepdims=True)
            q = np.where(tot > 0, sg / tot, 0.0) if c["norm"] else sg
            gz = (dw - (q * dw).sum(1, keepdims=True)) * q * (1 - sg) if c["norm"] else dw * sg * (1 - sg)
            np.add.at(dl, (t, ids[t, j]), 2.5 * gz[t, j])
        else:
            over = z if c["norm"] else l
            m = over.max(1, keepdims=True)
            m = np.where(np.isfinite(m), m, 0.0)
            den = np.exp(over - m).sum(1, keepdims=True)
            q = np.where(den > 0, np.exp(z - m) / den, 0.0)
            inner = (q * np.where(ids >= 0, dw, 0.0)).sum(1, keepdims=True)
            if not c["norm"]:
                dl -= 2.5 * inner * np.where(den > 0, np.exp(l - m) / den, 0.0)
            gz = q * (dw - inner) if c["norm"] else q * dw
            np.add.at(dl, (t, ids[t, j]), 2.5 * gz[t, j])
    return torch.from_numpy(2.5 * q), torch.from_numpy(dl)


def exact(case, seed):
    s = prepare(case, seed)
    c, op = s["c"], s["c"]["op"]
    if op == "route":
        l = s["logits"].float().cpu().numpy()
        key = l + s["bias"].cpu().numpy() if s["bias"] is not None else l
        ids = np.argsort(-key, axis=1, kind="stable")[:, : c["k"]]
        ids = np.where(np.take_along_axis(key, ids, 1) > -np.inf, ids, -1)
        return {"ids": None, "weights": _weights64(s, ids)[0], "rows": None, "src": None, "offs": None, "counts": None}
    if op == "route_grad":
        return _weights64(s, s["ids"].cpu().numpy())[1]
    if op in ("dispatch", "combine_grad"):
        T, k = s["rows"].shape
        t, j = (s["rows"] >= 0).nonzero(as_tuple=True)
        at = s["rows"][t, j].long()
        out = torch.zeros(s["out"].shape, dtype=torch.float64, device=DEV)
        x = s["x"].double()
        if op == "dispatch":
            out[at] = x[t]
            return out
        out[at] = x[t] * s["w"].double()[t, j][:, None]
        dw = torch.zeros((T, k), dtype=torch.float64, device=DEV)
        for i in range(0, t.numel(), 8192):
            u = slice(i, i + 8192)
            dw[t[u], j[u]] = (x[t[u]] * s["y"][at[u]].double()).sum(1)
        return {"dy": out, "dw": dw}
    if op == "combine":
        out = torch.zeros(s["out"].shape, dtype=torch.float64, device=DEV)
        t, j = (s["rows"] >= 0).nonzero(as_tuple=True)
        for jj in range(c["k"]):
            on = t[j == jj]
            out[on] += s["y"][s["rows"][on, jj].long()].double() * s["w"][on, jj].double()[:, None]
        return out
    if op == "glu":
        gu = _product64(s)
        F = c["F"]
        return {"h": _phi64(gu[:, :F], c["act"])[0] * gu[:, F:], "gu": gu if c["keep"] else None}
    if op == "glu_grad":
        dh, F = _product64(s), c["F"]
        a, da = _phi64(s["gu"][:, :F].double(), c["act"])
        return torch.cat([dh * s["gu"][:, F:].double() * da, dh * a], 1)
    if op == "glu_token":
        gu, F = _pairs64(s), c["F"]
        return _phi64(gu[:, :F], c["act"])[0] * gu[:, F:]
    if op == "down_token":
        return _pairs64(s)
    x, y = s["x"].double(), None
    y = x @ _lines64(s["b"][0][0], s["b"][1][0], s["b"][2]).T
    for a in range(c["n"]):
        at = (s["aid"] == a).nonzero().view(-1)
        y[at] += s["cs"][a].double() * ((x[at] @ s["A"][a].double().T) @ s["B"][a].double().T)
    return y

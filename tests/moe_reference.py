"""Plain 64-bit implementations of the operators in ``include/moe_ops.h`` on
the CPU, with the error bounds their tests use.  Written from the definitions;
nothing here calls the library."""
from __future__ import annotations

import numpy as np
import torch

FLT_MAX = float(np.finfo(np.float32).max)
U = 2.0 ** -24          # unit roundoff of fp32
UB = 2.0 ** -8          # unit roundoff of bf16 (8 significant bits)


# ------------------------------------------------------------------ NVFP4

E2M1 = np.array([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6])


def e4m3_table():
    c = np.arange(256)
    e, m = (c >> 3) & 15, c & 7
    return np.where(e == 0, m / 512.0, np.ldexp(1 + m / 8.0, e - 7))


def decode(data, scale):
    """value(code) * value(S) of lines: data [..., L, K/2], scale [..., L, K/16] -> f64 [..., L, K]."""
    data, scale = np.asarray(data), np.asarray(scale)
    v = np.empty((*data.shape, 2))
    v[..., 0], v[..., 1] = E2M1[data & 15], E2M1[data >> 4]
    return v.reshape(*data.shape[:-1], -1) * np.repeat(e4m3_table()[scale], 16, axis=-1)


def random_lines(rng, lines, k, big=1.0):
    """Random NVFP4 lines: codes, E4M3 scale bytes (zeros, subnormals and the largest among them) and amax."""
    data = rng.integers(0, 256, (lines, k // 2), dtype=np.uint8)
    scale = rng.integers(0x30, 0x7F, (lines, k // 16), dtype=np.uint8)
    scale[rng.random(scale.shape) < 0.05] = 0
    scale[rng.random(scale.shape) < 0.05] = 3
    amax = (big * np.exp(rng.standard_normal(lines))).astype(np.float32)
    if lines > 2:
        amax[rng.integers(lines)] = 0.0
    return data, scale, amax


def product(xa, sa, xb, sb):
    """sum_t xa xb with the lines' factors, and sum_t |xa xb| with them (for error bounds)."""
    f = sa[:, None] * sb[None, :]
    return (xa @ xb.T) * f, (np.abs(xa) @ np.abs(xb).T) * f


def gemm_bound(absum, k):
    """fp32 sum of k exact products, 2u per addition, and four roundings for the factors."""
    return (2 * k + 8) * U * absum


# --------------------------------------------------------------- routing

def clean(logits):
    l = np.asarray(logits, dtype=np.float64)
    return np.where(l > -np.inf, np.minimum(l, FLT_MAX), -np.inf)     # NaN compares false


def select(logits, k, bias=None):
    """ids [T, k]: the largest f32 keys, ties to the lower index, -1 where none is left."""
    l = clean(logits).astype(np.float32)
    with np.errstate(over="ignore"):
        key = l + bias.astype(np.float32) if bias is not None else l + np.float32(0)
    ids = np.argsort(-key.astype(np.float64), axis=1, kind="stable")[:, :k]
    return np.where(np.take_along_axis(key, ids, 1) > -np.inf, ids, -1).astype(np.int32)


def route_weights(logits, ids, score, normalize, scale):
    l = clean(logits)
    on = ids >= 0
    z = np.where(on, np.take_along_axis(l, np.maximum(ids, 0), 1), -np.inf)
    with np.errstate(all="ignore"):
        if score == "sigmoid":
            s = np.where(on, 1 / (1 + np.exp(-z)), 0.0)
        else:
            m = l.max(1, keepdims=True)
            m = np.where(np.isfinite(m), m, 0.0)
            tot = np.exp(l - m).sum(1, keepdims=True)
            s = np.where(on, np.exp(z - m) / np.where(tot > 0, tot, 1), 0.0)
            if normalize:   # over the chosen alone, which stays finite where their shares underflow
                mz = z.max(1, keepdims=True)
                s = np.where(on, np.exp(z - np.where(np.isfinite(mz), mz, 0.0)), 0.0)
        if normalize:
            t = s.sum(1, keepdims=True)
            s = np.where(t > 0, s / np.where(t > 0, t, 1), 0.0)
    return scale * s


def route_grad(logits, ids, dweights, score, normalize, scale):
    """d sum(weights * dweights) / d logits, from the formula of the weights."""
    l = clean(logits)
    T, E = l.shape
    on = ids >= 0
    on &= np.take_along_axis(l, np.maximum(ids, 0), 1) > -np.inf
    q = route_weights(logits, np.where(on, ids, -1), score, normalize, 1.0)
    g = np.where(on, scale * dweights, 0.0)
    z = np.where(on, np.take_along_axis(l, np.maximum(ids, 0), 1), -np.inf)
    dl = np.zeros((T, E))
    inner = (q * g).sum(1, keepdims=True)
    with np.errstate(all="ignore"):
        if score == "sigmoid":
            one_minus = np.where(on, 1 / (1 + np.exp(z)), 0.0)
            d = (g - inner if normalize else g) * q * one_minus
        elif normalize:
            d = q * (g - inner)
        else:
            m = l.max(1, keepdims=True)
            e = np.exp(l - np.where(np.isfinite(m), m, 0.0))
            t = e.sum(1, keepdims=True)
            dl = -inner * np.where(t > 0, e / np.where(t > 0, t, 1), 0.0)
            d = q * g
    t, j = np.nonzero(on)
    np.add.at(dl, (t, ids[t, j]), d[t, j])
    return dl


def plan(ids, E, cap):
    """counts, ends, rows, src of a flat list of choices."""
    ids = np.asarray(ids).reshape(-1)
    ok = (ids >= 0) & (ids < E)
    counts = np.bincount(ids[ok], minlength=E).astype(np.int64)
    padded = (counts + 127) // 128 * 128
    ends = np.cumsum(padded)
    at = ends - padded
    rows, src = np.full(ids.size, -1, np.int64), np.full(cap, -1, np.int64)
    for p in np.nonzero(ok)[0]:
        r = at[ids[p]]
        at[ids[p]] += 1
        if r < cap:
            rows[p] = r
            src[r] = p
    return counts, ends, rows, src


# ------------------------------------------------------------- activation

def act(g, kind):
    """act(g), act'(g) and bounds on |act'| and |act''|."""
    if kind == "silu":
        q = 1 / (1 + np.exp(-g))
        return g * q, q + g * q * (1 - q)
    # (1 + tanh(w)) / 2 as the logistic of 2w: 1 + tanh(w) cancels for negative w
    w2 = 2 * np.sqrt(2 / np.pi) * (g + 0.044715 * g ** 3)
    with np.errstate(over="ignore"):
        q, r = 1 / (1 + np.exp(-w2)), 1 / (1 + np.exp(w2))
    return g * q, q + g * q * r * 2 * np.sqrt(2 / np.pi) * (1 + 3 * 0.044715 * g ** 2)


# The logistic q = rcp(1 + exp(-v)) in fp32: v's rounding (a few u relative)
# moves e^-v by |v| times that, the hardware exponential and reciprocal add at
# most 4 u each; where e^-v dominates the relative error of q is theirs in full.
def act_rel(g, kind):
    v = np.abs(g) if kind == "silu" else np.minimum(1.6 * np.abs(g) * (1 + 0.045 * g ** 2), 200.0)
    return (6 * v + 16) * U


def glu_bound(g, u, dg, du, kind):
    """|h - exact| for h = act(g) u with errors dg, du in g and u, rounded to bf16."""
    a, _ = act(g, kind)
    h = np.abs(a * u)
    e = 1.2 * dg * np.abs(u) + (np.abs(a) + 1.2 * dg) * du + h * act_rel(g, kind) + 1e-30
    return e + UB * (h + e) + 2.0 ** -134


def to_dev(a):
    a = np.ascontiguousarray(a)
    return torch.from_numpy(a).to("cuda:0")


def bf16_round(a):
    """fp32/64 values rounded to bf16, as a torch tensor and as f64 numpy."""
    t = torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).to(torch.bfloat16)
    return t, t.double().numpy()


def check(got, want, bound, what):
    got = got.double().cpu().numpy() if isinstance(got, torch.Tensor) else np.asarray(got, np.float64)
    assert got.shape == want.shape, (what, got.shape, want.shape)
    assert np.isfinite(got).all(), what
    over = np.abs(got - want) - bound
    i = np.unravel_index(np.argmax(over), over.shape) if over.size else None
    assert not over.size or over[i] <= 0, f"{what}: at {i} got {got[i]} want {want[i]} bound {np.broadcast_to(bound, want.shape)[i]}"

"""Plain implementations, on the CPU and from the definitions, of the operators
in ``include/i8_group.h`` and of the balance loss and the 8-bit checkpoint in
``include/moe_ops.h``; nothing here calls the library."""
from __future__ import annotations

import numpy as np
import torch

import moe_reference as R

F = np.float32


# ------------------------------------------------------------ 8-bit integers

def cast(x):
    """Codes and scales of rows of bf16 values (given as fp32), each step one fp32 operation."""
    x = np.asarray(x, F)
    with np.errstate(all="ignore"):
        amax = np.abs(x).max(1, keepdims=True)
        bad = ~np.isfinite(x).all(1, keepdims=True)
        pre = np.where(amax < F(2.0 ** -100), F(2.0 ** 64), F(1)).astype(F)
        inv = np.where(amax > 0, F(127) / (amax * pre), F(0)).astype(F)
        q = np.rint((x * pre) * inv)
    q = np.where(bad, 0, q).astype(np.int8)
    return q, np.where(bad, F(np.nan), amax / F(127)).astype(F)[:, 0]


def random_codes(rng, *shape):
    """Codes over the whole range, -128 and 127 often."""
    q = rng.integers(-128, 128, shape, dtype=np.int8)
    q[rng.random(shape) < 0.1] = -128
    q[rng.random(shape) < 0.1] = 127
    return q


def product(qa, sa, qb, sb):
    """The exact sum as fp32, times the row's, then times the channel's scale: fp32 [rows, lines]."""
    acc = qa.astype(np.float64) @ qb.astype(np.float64).T            # below 2^53: exact
    with np.errstate(all="ignore"):
        return (acc.astype(F) * sa[:, None].astype(F)) * sb[None, :].astype(F)


def grouped(qa, sa, qb, sb, splits):
    out, at = [], 0
    for e, m in enumerate(splits):
        out.append(product(qa[at:at + m], sa[at:at + m], qb[e], sb[e]))
        at += m
    return np.concatenate(out)


def same_bits(got, want, what):
    """got (fp32 or bf16 tensor) holds want (fp32), rounded once to its type; NaN where want is."""
    got = got.cpu()
    want = torch.from_numpy(np.ascontiguousarray(want)).to(got.dtype)
    nan = torch.isnan(want)
    assert got.shape == want.shape, (what, got.shape, want.shape)
    assert torch.equal(torch.isnan(got), nan), what
    bad = (got != want) & ~nan
    assert not bad.any(), f"{what}: {int(bad.sum())} differ, first at {bad.nonzero()[0].tolist()}"


# -------------------------------------------------------------- balance loss

def probabilities(logits, score):
    """p and 1 - s (1 for softmax), f64; 0 where masked."""
    l = R.clean(logits)
    on = l > -np.inf
    with np.errstate(all="ignore"):
        if score == "sigmoid":
            s = np.where(on, 1 / (1 + np.exp(-l)), 0.0)
            slope = np.where(on, 1 / (1 + np.exp(l)), 1.0)
        else:
            m = l.max(1, keepdims=True)
            s = np.where(on, np.exp(l - np.where(np.isfinite(m), m, 0.0)), 0.0)
            slope = np.ones_like(s)
    t = s.sum(1, keepdims=True)
    return np.where(t > 0, s / np.where(t > 0, t, 1), 0.0), slope, on.any(1)


def balance(logits, ids, ends, score, coef, topk):
    """loss, counts, probs, tokens and the gradient in the logits (for dloss 1)."""
    T, E = logits.shape
    ends = [T] if ends is None else list(ends)
    S = len(ends)
    p, slope, any_ = probabilities(logits, score)
    counts, probs, tokens = np.zeros((S, E), np.int64), np.zeros((S, E)), np.zeros(S, np.int64)
    grad, scale = np.zeros((T, E)), np.zeros((T, 1))
    loss, b = 0.0, 0
    for s, e in enumerate(ends):
        c = ids[b:e].reshape(-1)
        counts[s] = np.bincount(c[(c >= 0) & (c < E)], minlength=E)
        probs[s], tokens[s] = p[b:e].sum(0), int(any_[b:e].sum())
        if tokens[s]:
            w = coef / S * E / (topk * float(tokens[s]) ** 2)
            a = w * counts[s]
            loss += float(a @ probs[s])
            inner = p[b:e] @ a
            grad[b:e] = p[b:e] * slope[b:e] * (a - inner[:, None])
            # what an error of p counts against: every term of the two products
            scale[b:e, 0] = abs(w) * (np.abs(counts[s]).max() + p[b:e] @ np.abs(counts[s]))
        b = e
    return loss, counts, probs, tokens, grad, p * slope * scale


def balance_bounds(logits, ids, ends, score, coef, topk, rel):
    """What probs and the loss may be off by, from the depth of their sums and not from their length.  rel [T, E]: the
    relative error of a sigmoid or exponential.  All terms are positive, so a sum is off by its terms' errors and one u
    for each addition that a term goes through: of probs at most 32 rows of a lane, 3 exchanges, 16 waves, 8 slots of a
    joining part, an exchange and 16 waves (80 u); of the loss also the product with the count, 6 exchanges (16 experts
    of a thread and 16 waves where one work-group does it all, without a join), 7 roundings of the weight, up to 128
    shares of a thread, 6 exchanges and 16 waves (256 u)."""
    p, _, any_ = probabilities(logits, score)
    T, E = logits.shape
    each = p * (rel + (p * rel).sum(1, keepdims=True))        # its own error, and that of the sum it is divided by
    loss, counts, probs, tokens, _, _ = balance(logits, ids, ends, score, coef, topk)
    ends = [T] if ends is None else list(ends)
    off, loss_off, b = np.zeros((len(ends), E)), 256 * R.U * loss + 1e-37, 0
    for s, e in enumerate(ends):
        if tokens[s]:
            off[s] = each[b:e].sum(0) + 80 * R.U * probs[s] + tokens[s] * 1e-37
            loss_off += coef / len(ends) * E / (topk * float(tokens[s]) ** 2) * float(counts[s] @ off[s])
        b = e
    return off, loss_off


# ----------------------------------------------------------- 8-bit checkpoint

def group_of(f):
    """Scale group of each column of g (then of u)."""
    g = np.arange(f) // 32
    return np.concatenate([g, g + -(-f // 32)])


def kept_values(codes, scales, f):
    """f64 values [M, 2f] of codes [M, 2f] and bf16 scales [groups, M]."""
    s = scales.double().cpu().numpy().T[:, group_of(f)]
    return codes.cpu().numpy().astype(np.float64) * s, s

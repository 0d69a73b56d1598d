"""Inputs, oracle values and tolerances of the expert-parallel tests."""

import numpy as np
import torch

from oracle import experts as X

TORCH = {"float32": torch.float32, "bfloat16": torch.bfloat16, "int32": torch.int32, "int64": torch.int64}
# Half a step of the stored type, relative to the value.
HALF = {"float32": 2.0 ** -24, "bfloat16": 2.0 ** -8}
EPS = 2.0 ** -23  # a float32 step: one operation of a sum, whichever way the unit rounds


def choices(rng, n, tokens, topk, experts, padded=0.1):
    """Router choices with repeats, some experts never chosen, some padding
    (-1) and some numbers outside [0, experts)."""
    popular = rng.permutation(experts)[:max(1, (3 * experts + 3) // 4)]
    ids = rng.choice(popular, size=(n, tokens, topk)).astype(np.int32)
    ids[rng.random(ids.shape) < padded] = -1
    ids[rng.random(ids.shape) < padded / 4] = experts + 7
    return ids


def route_sorted(ids, experts, capacity):
    """X.route by one stable sort, for many choices."""
    n, per_rank = ids.shape[0], experts // ids.shape[0]
    flat = ids.reshape(-1).astype(np.int64)
    key = np.where((flat >= 0) & (flat < experts), flat, experts)
    order = np.argsort(key, kind="stable")
    ends = np.cumsum(np.bincount(key, minlength=experts + 1)[:experts])
    starts = np.concatenate([[0], ends])[::per_rank]  # rows of the ranks before; of all, for no choice
    rank = key // per_rank
    row = np.empty_like(key)
    row[order] = np.arange(len(key))
    row -= starts[np.minimum(rank, n)]
    places = np.where((key < experts) & (row < capacity), rank * capacity + row, -1)
    offsets = np.minimum(np.concatenate([np.zeros((n, 1), np.int64), ends.reshape(n, -1) - starts[:n, None]], 1), capacity)
    return places.reshape(ids.shape).astype(np.int32), offsets.astype(np.int32)


def values(rng, shape, dtype, scale=1.0):
    """Normal values as the stored type holds them: (float64 array, device tensor maker)."""
    v = torch.from_numpy((rng.standard_normal(shape) * scale).astype(np.float32)).to(TORCH[dtype])
    return v.double().numpy(), v


def ranges(rng, n, per_rank, capacity, empty=0.25):
    """Offsets [n, per_rank + 1]: random cuts of up to `capacity` rows, some experts empty."""
    off = np.zeros((n, per_rank + 1), np.int32)
    for r in range(n):
        share = rng.random(per_rank) * (rng.random(per_rank) > empty)
        total = int(rng.integers(0, capacity + 1))
        if share.sum() > 0:
            off[r, 1:] = np.floor(np.cumsum(share) / share.sum() * total + 1e-9)
    return off


def shifted(t, offset):
    """A copy of the tensor `offset` elements into a larger allocation."""
    big = torch.empty(t.numel() + offset + 8, dtype=t.dtype, device="cuda")
    view = big[offset:offset + t.numel()].view(t.shape)
    view.copy_(t)
    return view


def check(got, want, bound, what):
    """|got - want| <= bound everywhere, and no value that is not a number."""
    got = got.detach().double().cpu().numpy()
    assert got.shape == want.shape, (what, got.shape, want.shape)
    off = np.abs(got - want)
    bad = ~(off <= bound)
    if bad.any():
        at = tuple(int(i[0]) for i in np.nonzero(bad))
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.size} off, first at {at}: got {got[at]!r}, want "
                             f"{want[at]!r}, bound {np.broadcast_to(bound, want.shape)[at]!r}")


def sum_bound(size, terms, dtype, want):
    """A float32 sum of `terms` products whose sizes add up to `size`, rounded
    once to dtype: each of the terms + 1 operations is off by at most a step
    of the running sum, which is at most `size`."""
    error = (terms + 2) * EPS * size
    return error + HALF[dtype] * (np.abs(want) + error)


def product_bound(z, size, terms, dtype, activation, residual, want):
    """As sum_bound, through an activation.  Its slope is at most 1.13 (GELU;
    SiLU 1.10), so it passes on at most 1.13 of z's error; its own float32
    evaluation (erf, exp, divisions and products, a few steps each) is off by
    at most 16 steps of |z| + 1, the residual's sum by one of its result."""
    error = 1.13 * (terms + 2) * EPS * size
    if activation in ("gelu", "silu"):
        error = error + 16 * EPS * (np.abs(z) + 1)
    if residual is not None:
        error = error + EPS * (np.abs(want) + error)
    return error + HALF[dtype] * (np.abs(want) + error)


def grad_bound(size, terms, dtype, activation, want):
    """A sum of products with dz: its float32 evaluation is off by at most 32
    steps of |g|·(1 + |z|) (size counts |dz|, and where the slope is small a
    step of the slope's terms counts: see the callers' `floor`), and a bf16 dz
    is rounded, half a step a term."""
    error = (terms + 2) * EPS * size
    if activation != "none":
        error = error + (HALF[dtype] if dtype == "bfloat16" else 0.0) * size
    return error + HALF[dtype] * (np.abs(want) + error)


__all__ = ["X", "np", "torch", "TORCH", "HALF", "EPS", "choices", "route_sorted", "values", "ranges", "shifted", "check", "sum_bound",
           "product_bound", "grad_bound"]

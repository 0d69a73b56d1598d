"""The expert-parallel calls without a GPU: refusals before any HIP call
(device addresses are fake integers, never dereferenced), workspace sizes,
and the oracle against brute force, autograd and differences."""

import ctypes
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

from oracle import experts as X

BASE = 1 << 33


@pytest.fixture(scope="module")
def cs():
    from collective_reduction_amd import ccl_sim
    return ccl_sim


def fake(n, slot, step=1 << 24):
    """Addresses of n rank buffers, disjoint from those of other slots."""
    return [BASE + (slot << 36) + r * step for r in range(n)]


SIZES = {"nranks": 2, "experts": 4, "topk": 2, "tokens": 8, "capacity": 10, "hidden": 16, "features": 24}


def call(cs, op, shape=None, workspace="own", dtype="float32", **over):
    """One call with valid fake arguments, some of them replaced."""
    sizes = {**SIZES, **(shape or {})}
    s = cs.ExpertShape(**sizes)
    n = max(sizes["nranks"], 1)
    kw = {
        "route": dict(ids=fake(n, 1), places=fake(n, 2), offsets=fake(n, 3)),
        "dispatch": dict(sendbufs=fake(n, 1), places=fake(n, 2), recvbufs=fake(n, 3)),
        "combine": dict(sendbufs=fake(n, 1), places=fake(n, 2), recvbufs=fake(n, 3), weights=fake(n, 4), residual=fake(n, 5)),
        "combine_grad": dict(grads=fake(n, 1), places=fake(n, 2), sendbufs=fake(n, 3), weights=fake(n, 4),
                             grad_rows=fake(n, 5), grad_weights=fake(n, 6)),
        "matmul": dict(rows=fake(n, 1), weights=fake(n, 2), out=fake(n, 3), offsets=fake(n, 4), bias=fake(n, 5),
                       residual=fake(n, 6), preact=fake(n, 7), activation="silu"),
        "matmul_grad": dict(grads=fake(n, 1), rows=fake(n, 2), weights=fake(n, 3), offsets=fake(n, 4), preact=fake(n, 5),
                            activation="silu", grad_rows=fake(n, 6), grad_weights=fake(n, 7), grad_bias=fake(n, 8)),
    }[op]
    kw.update(over)
    if workspace == "own":
        workspace = (BASE << 8, 1 << 40)
    if op == "route" and dtype == "float32":
        dtype = "int32"
    getattr(cs, "ccl_sim_expert_" + op)(s, workspace=workspace, dtype=dtype, **kw)


def refused(cs, op, code=None, match=None, **kw):
    with pytest.raises(cs.CclSimError, match=match) as e:
        call(cs, op, **kw)
    assert e.value.code == (cs.INVALID_ARGUMENT if code is None else code)


OPS = ("route", "dispatch", "combine", "combine_grad", "matmul", "matmul_grad")


@pytest.mark.parametrize("op", OPS)
def test_shapes_out_of_range_are_refused(cs, op):
    for nranks in (0, -1, 1025):
        refused(cs, op, shape={"nranks": nranks})
    refused(cs, op, match="2\\^31", shape={"capacity": 1 << 30})
    refused(cs, op, match="2\\^31", shape={"capacity": (1 << 64) - 1})
    if op in ("route", "matmul", "matmul_grad"):
        for experts in (0, 3, 2050, -2):
            refused(cs, op, match="experts", shape={"experts": experts})
    if not op.startswith("matmul"):
        for topk in (0, 65, -1):
            refused(cs, op, match="topk", shape={"topk": topk})
        refused(cs, op, match="2\\^31", shape={"tokens": 1 << 29})
        refused(cs, op, match="2\\^31", shape={"tokens": 1 << 63})
    if op != "route":
        refused(cs, op, match="hidden", shape={"hidden": (1 << 20) + 1})
    if op.startswith("matmul"):
        refused(cs, op, match="features", shape={"features": (1 << 20) + 1})
        refused(cs, op, match="hidden=0", shape={"hidden": 0})
        refused(cs, op, match="one launch", shape={"hidden": 1 << 20, "features": 1 << 20})
    with pytest.raises(ValueError, match="ExpertShape"):
        getattr(cs, "ccl_sim_expert_" + op)((2, 4), *[fake(2, 1)] * 3)


def test_types_are_checked(cs):
    for dtype in ("float32", "bfloat16"):
        with pytest.raises(cs.CclSimError, match="int32 or int64"):
            cs.ccl_sim_expert_route(cs.ExpertShape(**SIZES), fake(2, 1), fake(2, 2), fake(2, 3), dtype=dtype)
    for op in ("combine", "combine_grad", "matmul", "matmul_grad"):
        for dtype in ("int32", "int64"):
            refused(cs, op, match="float32 and bf16", dtype=dtype)
    refused(cs, "dispatch", dtype=9)
    for op in ("matmul", "matmul_grad"):
        refused(cs, op, match="activation", activation=4)
        with pytest.raises(ValueError, match="activation"):
            call(cs, op, activation="tanh")


POINTERS = [(op, name) for op, names in (
    ("route", ("ids", "places", "offsets")), ("dispatch", ("sendbufs", "places", "recvbufs")),
    ("combine", ("sendbufs", "places", "recvbufs", "weights", "residual")),
    ("combine_grad", ("grads", "places", "sendbufs", "weights", "grad_rows", "grad_weights")),
    ("matmul", ("rows", "weights", "out", "offsets", "bias", "residual", "preact")),
    ("matmul_grad", ("grads", "rows", "weights", "offsets", "preact", "grad_rows", "grad_weights", "grad_bias")),
) for name in names]


@pytest.mark.parametrize("op,name", POINTERS)
def test_pointers_are_checked(cs, op, name):
    refused(cs, op, match=rf"{name}\[1\] is NULL", **{name: [BASE, 0]})
    refused(cs, op, match=rf"{name}\[0\] is not aligned", **{name: [BASE + 1, BASE + (1 << 24)]})
    with pytest.raises(ValueError, match="ranks"):
        call(cs, op, **{name: fake(3, 9)})


@pytest.mark.parametrize("op,out,others", [
    ("route", "places", ("ids", "offsets")), ("route", "offsets", ("ids",)),
    ("dispatch", "recvbufs", ("sendbufs", "places")), ("combine", "recvbufs", ("sendbufs", "places", "weights")),
    ("combine_grad", "grad_rows", ("grads", "places", "sendbufs", "weights", "grad_weights")),
    ("combine_grad", "grad_weights", ("grads", "places", "sendbufs", "weights")),
    ("matmul", "out", ("rows", "weights", "offsets", "bias", "preact")),
    ("matmul", "preact", ("rows", "weights", "offsets", "bias", "residual")),
    ("matmul_grad", "grad_rows", ("grads", "rows", "weights", "offsets", "preact", "grad_weights", "grad_bias")),
    ("matmul_grad", "grad_weights", ("grads", "rows", "weights", "offsets", "preact", "grad_bias")),
    ("matmul_grad", "grad_bias", ("grads", "rows", "weights", "offsets", "preact")),
])
def test_overlapping_buffers_are_refused(cs, op, out, others):
    for name in others:
        refused(cs, op, match="overlap", **{out: fake(2, 20), name: [v + 8 for v in fake(2, 20)]})
        refused(cs, op, match="overlap", **{out: fake(2, 20), name: fake(2, 20)[::-1]})
    refused(cs, op, match="overlap", **{out: [BASE + (20 << 36), BASE + (20 << 36)]})
    if op in ("route",):
        return
    ws = (fake(2, 20)[1] // 256 * 256, 1 << 40)
    if cs.ccl_sim_expert_workspace_size(op, cs.ExpertShape(**SIZES)):
        refused(cs, op, match="workspace overlaps", workspace=ws, **{out: fake(2, 20)})


def test_residual_in_place_is_for_the_same_rank_only(cs):
    for op, out in (("combine", "recvbufs"), ("matmul", "out")):
        refused(cs, op, match="overlap", **{out: fake(2, 20), "residual": [v + 16 for v in fake(2, 20)]})
        refused(cs, op, match="overlap", **{out: fake(2, 20), "residual": fake(2, 20)[::-1]})


def test_workspace_is_checked(cs):
    need = cs.ccl_sim_expert_workspace_size("matmul_grad", cs.ExpertShape(**SIZES))
    assert need >= 2 * 10 * 24 * 4
    refused(cs, "matmul_grad", cs.INSUFFICIENT_WORKSPACE, workspace=None)
    refused(cs, "matmul_grad", cs.INSUFFICIENT_WORKSPACE, workspace=(BASE << 8, need - 1))
    refused(cs, "matmul_grad", match="256-byte", workspace=((BASE << 8) + 64, need))
    many = {"nranks": 65, "experts": 65}
    for op in OPS:
        refused(cs, op, cs.INSUFFICIENT_WORKSPACE, workspace=None, shape=many)


def test_workspace_sizes(cs):
    size = cs.ccl_sim_expert_workspace_size
    invalid = ctypes.c_size_t(-1).value
    s = cs.ExpertShape(**SIZES)
    assert size("route", s) == 0 and size("dispatch", s, "int64") == 0
    assert size("combine", s, "bfloat16") == 0 and size("combine_grad", s, "bfloat16") == 0
    assert size("matmul", s, "int32") == invalid and size(6, s) == invalid
    assert size("route", cs.ExpertShape(**{**SIZES, "experts": 3})) == invalid
    assert "experts=3" in cs.ccl_sim_last_error()
    long = cs.ExpertShape(**{**SIZES, "tokens": 100_000})
    assert size("route", long) >= 4 * 4 * (400_000 // 4096)
    with pytest.raises(ValueError, match="experts=3"):
        cs.ExpertWorkspace("route", cs.ExpertShape(**{**SIZES, "experts": 3}), device="cpu")


def test_offsets_may_be_left_out_for_one_expert_a_rank_only(cs):
    refused(cs, "matmul", match="one expert per rank", offsets=None)
    refused(cs, "matmul_grad", match="one expert per rank", offsets=None)


def test_empty_calls_succeed_with_null_pointers(cs):
    nobody = [0, 0]
    for sizes in ({"tokens": 0}, {"hidden": 0}, {"capacity": 0}):
        call(cs, "dispatch", shape=sizes, sendbufs=nobody, places=nobody, recvbufs=nobody)
    for sizes in ({"tokens": 0}, {"hidden": 0}):
        call(cs, "combine", shape=sizes, sendbufs=nobody, places=nobody, recvbufs=nobody, weights=None, residual=None)
    call(cs, "combine_grad", shape={"tokens": 0}, grads=nobody, places=nobody, sendbufs=nobody, weights=nobody,
         grad_rows=nobody, grad_weights=nobody)
    for sizes in ({"capacity": 0}, {"features": 0}):
        call(cs, "matmul", shape=sizes, rows=nobody, weights=nobody, out=nobody, offsets=nobody, bias=nobody,
             residual=nobody, preact=nobody)
    call(cs, "matmul_grad", grad_rows=None, grad_weights=None, grad_bias=None)


ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("empty,absent,asked", [
    ("capacity", ("rows", "grads", "preact"), "grad_weights"), ("capacity", ("rows", "grads", "weights"), "grad_bias"),
    ("features", ("weights", "grads", "preact"), "grad_rows")])
def test_gradients_of_nothing_read_no_array_that_is_null(empty, absent, asked):
    """Arrays of no elements may be NULL: the call gets as far as a machine
    without a GPU lets it.  In a process of its own, with no GPU to be seen."""
    code = f"""
import test_experts_cpu as t
from collective_reduction_amd import ccl_sim as cs
outputs = {{k: None for k in ("grad_rows", "grad_weights", "grad_bias") if k != {asked!r}}}
try:
    t.call(cs, "matmul_grad", shape={{{empty!r}: 0}}, **{{k: None for k in {absent!r}}}, **outputs)
except cs.CclSimError as e:
    assert e.code == cs.HIP_ERROR, e
print("returned")
"""
    paths = os.pathsep.join((ROOT, os.path.join(ROOT, "tests")))
    env = {**os.environ, "HIP_VISIBLE_DEVICES": "-1", "PYTHONPATH": paths}
    done = subprocess.run([sys.executable, "-c", code], env=env, capture_output=True, text=True, timeout=300)
    assert done.returncode == 0 and done.stdout.strip().endswith("returned"), (done.returncode, done.stderr[-500:])


def test_binding_checks_tensors(cs):
    s = cs.ExpertShape(**SIZES)
    host = torch.zeros(2, 8, 16)
    places = torch.zeros(2, 8, 2, dtype=torch.int32)
    with pytest.raises(ValueError, match="device buffers"):
        cs.ccl_sim_expert_dispatch(s, host, places, torch.zeros(2, 10, 16))
    with pytest.raises(ValueError, match="first dimension is the rank"):
        cs.ccl_sim_expert_dispatch(s, torch.zeros(3, 8, 16), places, host)
    with pytest.raises(ValueError, match="not contiguous"):
        cs.ccl_sim_expert_dispatch(s, torch.zeros(16, 8, 2).transpose(0, 2), places, host)
    with pytest.raises(ValueError, match="unknown expert operator"):
        cs.ExpertPlan("scatter", s)


# --------------------------------------------------------------------------
# the oracle
# --------------------------------------------------------------------------

def small_case(seed):
    rng = np.random.default_rng(seed)
    n, per_rank, topk, tokens, capacity = 3, 2, 2, 5, 7
    ids = rng.integers(-1, n * per_rank, (n, tokens, topk)).astype(np.int32)
    return rng, ids, n, per_rank, topk, tokens, capacity


@pytest.mark.parametrize("seed", range(4))
def test_oracle_route_is_a_stable_sort(seed):
    _, ids, n, per_rank, topk, tokens, capacity = small_case(seed)
    places, offsets = X.route(ids, n * per_rank, capacity)
    flat = ids.reshape(-1)
    for d in range(n):
        chosen = [a for a in np.argsort(flat, kind="stable") if d * per_rank <= flat[a] < (d + 1) * per_rank]
        for row, a in enumerate(chosen):
            assert places.reshape(-1)[a] == (d * capacity + row if row < capacity else -1)
        for e in range(per_rank + 1):
            assert offsets[d, e] == min(capacity, sum(flat[a] < d * per_rank + e for a in chosen))
    assert (places[ids < 0] == -1).all()


@pytest.mark.parametrize("n,experts,topk,tokens,capacity", [(3, 6, 2, 5, 7), (1, 9, 3, 40, 30), (4, 4, 1, 50, 60), (2, 8, 2, 0, 3)])
def test_route_by_sort_is_the_oracles(n, experts, topk, tokens, capacity):
    from expert_util import choices, route_sorted
    ids = choices(np.random.default_rng([n, experts, tokens]), n, tokens, topk, experts)
    for got, want in zip(route_sorted(ids, experts, capacity), X.route(ids, experts, capacity)):
        assert got.dtype == want.dtype and np.array_equal(got, want)


def test_oracle_exchange_round_trip_and_gradients_by_differences():
    rng, ids, n, per_rank, topk, tokens, capacity = small_case(9)
    places, _ = X.route(ids, n * per_rank, capacity)
    x, w = rng.standard_normal((n, tokens, 4)), rng.random((n, tokens, topk))
    rows = X.dispatch(x, places, np.zeros((n, capacity, 4)))
    kept = (places >= 0).sum(-1)[..., None]
    assert np.allclose(X.combine(rows, places), x * kept)
    y, g = rng.standard_normal((n, capacity, 4)), rng.standard_normal((n, tokens, 4))
    grad_rows, grad_weights = X.combine_grad(g, y, places, w)
    loss = lambda y, w: (X.combine(y, places, w) * g).sum()  # noqa: E731
    h = 1e-6
    for at in [(0, 0, 0), (1, 2, 3), (2, 6, 1)]:
        up, down = y.copy(), y.copy()
        up[at] += h
        down[at] -= h
        assert abs((loss(up, w) - loss(down, w)) / (2 * h) - grad_rows[at]) < 1e-7
    for at in [(0, 0, 0), (1, 4, 1), (2, 2, 0)]:
        up, down = w.copy(), w.copy()
        up[at] += h
        down[at] -= h
        assert abs((loss(y, up) - loss(y, down)) / (2 * h) - grad_weights[at]) < 1e-7


@pytest.mark.parametrize("activation", ["none", "relu", "gelu", "silu"])
def test_oracle_products_against_autograd_and_differences(activation):
    rng = np.random.default_rng(3)
    n, per_rank, capacity, hidden, features = 2, 3, 9, 5, 4
    off = np.array([[0, 4, 4, 7], [0, 0, 9, 9]], np.int32)
    x, w, b = (rng.standard_normal(s) for s in ((n, capacity, hidden), (n, per_rank, features, hidden), (n, per_rank, features)))
    res, g = rng.standard_normal((n, capacity, features)), rng.standard_normal((n, capacity, features))
    tx, tw, tb = (torch.from_numpy(v).requires_grad_() for v in (x, w, b))
    act = {"none": lambda z: z, "relu": torch.relu, "gelu": torch.nn.functional.gelu, "silu": torch.nn.functional.silu}[activation]
    loss = 0.0
    out, z, _ = X.matmul(x, off, w, b, res, activation)
    for r in range(n):
        for e in range(per_rank):
            lo, hi = off[r, e], off[r, e + 1]
            y = act(tx[r, lo:hi] @ tw[r, e].T + tb[r, e]) + torch.from_numpy(res[r, lo:hi])
            assert np.allclose(out[r, lo:hi], y.detach().numpy())
            loss = loss + (y * torch.from_numpy(g[r, lo:hi])).sum()
    want = torch.autograd.grad(loss, (tx, tw, tb))
    got = X.matmul_grad(g, x, off, w, z, activation)
    for name, v in zip(("rows", "weights", "bias"), want):
        assert np.allclose(got[name][0], v.numpy()), name
    value = lambda w: (X.matmul(x, off, w, b, res, activation)[0] * g * (np.arange(capacity)[None, :] < off[:, -1:])[..., None]).sum()  # noqa: E731
    for at in [(0, 0, 1, 2), (1, 1, 3, 0)]:
        up, down = w.copy(), w.copy()
        up[at] += 1e-6
        down[at] -= 1e-6
        assert abs((value(up) - value(down)) / 2e-6 - got["weights"][0][at]) < 1e-6

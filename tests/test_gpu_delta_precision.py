"""The bits that the delta rule keeps in bf16, on the GPU.

Differences that only whole operands leave: each call below is made so that one entry of a result is the difference of
two sums of 1 + 2^-9 and more, one of them 2^-20 larger.  Every product and sum on the way to it is exact in fp32 in any
order (at most 21 bits), so the entry has to be exact; with an operand held in 16 bits, two bf16 parts (1 and 2^-9), it
would be 0.

Random values: an element is off by half a step of its storage type and by fp32 roundings, which delta_reference.py
derives for results of fp32, element by element and in the 2-norm.
"""
import numpy as np
import pytest

from delta_reference import gradient_terms, make, values
from oracle import delta
from test_gpu_delta import CASES, _dev, _host, _lib, packed
from test_gpu_delta_backward import CASES as GRADIENT_CASES, run

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

A, B, E = 2.0 ** -3, 2.0 ** -6, 2.0 ** -10   # (1, A, E) . (1, B, E) = 1 + 2^-9 + 2^-20
LONG, SHORT = 1 + 2.0 ** -9 + 2.0 ** -20, 1 + 2.0 ** -9


def _zeros(T, K=40, V=24):
    """q, k, v, g, beta, state, do, dstate of one head, all 0, as arrays that a case fills in."""
    return {"q": np.zeros((T, 1, K)), "k": np.zeros((T, 1, K)), "v": np.zeros((T, 1, V)), "g": np.zeros((T, 1)),
            "b": np.zeros((T, 1)), "st": np.zeros((1, 1, K, V)), "do": np.zeros((T, 1, V)), "dl": np.zeros((1, 1, K, V))}


def _state(x):
    """o = h' q, h in 24 bits."""
    x["st"][0, 0, 5, 7], x["st"][0, 0, 33, 7] = LONG, SHORT
    x["q"][2, 0, [5, 33]] = 1, -1
    return 2, 7


def _scores(x):
    """o_40 = P u_0 + P u_1, P in 24 bits; the second token's value makes its u 1."""
    x["k"][0, 0, [0, 1, 35]] = 1, A, E
    x["k"][1, 0, [0, 1]] = -1, -A
    x["v"][0, 0], x["v"][1, 0], x["b"][:2] = 1, -(A * A), 1
    x["q"][40, 0, [0, 1, 35]] = 1, B, E
    return 40, 3


def _replaced(x):
    """o_20 = u_0 - u_1, u in 24 bits by beta."""
    x["k"][0, 0, 3] = x["k"][1, 0, 38] = 1
    x["v"][:2, 0], x["b"][0], x["b"][1] = 1, LONG, SHORT
    x["q"][20, 0, [3, 38]] = 1, -1
    return 20, 11


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("case", [_state, _scores, _replaced], ids=lambda f: f.__name__[1:])
def test_outputs_of_whole_operands(case, dtype):
    x = _zeros(41)
    t, c = case(x)
    args = tuple(x[n] for n in ("q", "k", "v", "g", "b", "st"))
    want = delta.delta_rule(*args[:5], [41], args[5])[0]
    assert want[t, 0, c] == 2.0 ** -20
    got = _host(packed(args, [41], dtype)[0])
    assert got[t, 0, c] == 2.0 ** -20


def _behind(x):
    """dk = D u, D in 24 bits."""
    x["dl"][0, 0, 5, [3, 20]] = LONG, -SHORT
    x["v"][0, 0], x["b"][0] = 1, 1
    return "dk", 0, 5


def _replaced_back(x):
    """dk = D u, u in 24 bits by the state."""
    x["k"][0, 0, 0] = 1
    x["st"][0, 0, 0, [3, 20]] = 1 - LONG, 1 - SHORT
    x["v"][0, 0], x["b"][0] = 1, 1
    x["dl"][0, 0, 33, [3, 20]] = 1, -1
    return "dk", 0, 33


def _before(x):
    """dk = -H dz, H in 24 bits."""
    x["k"][0, 0, 0], x["b"][0] = 1, 1
    x["st"][0, 0, 1, [3, 20]] = LONG, -SHORT
    x["dl"][0, 0, 0, [3, 20]] = 1
    return "dk", 0, 1


def _errors(x):
    """dk = -H dz, dz in 24 bits."""
    x["k"][0, 0, 0], x["b"][0] = 1, 1
    x["st"][0, 0, 1, [3, 20]] = 1, -1
    x["dl"][0, 0, 0, [3, 20]] = LONG, SHORT
    return "dk", 0, 1


def _values_seen(x):
    """dk_0 = sum over later tokens of (do . u_0) q, the factors in 24 bits."""
    x["v"][0, 0, [0, 1, 20]], x["b"][0] = (1, A, E), 1
    x["do"][1, 0, [0, 1, 20]] = 1, B, E
    x["do"][30, 0, [0, 1]] = 1, B
    x["q"][1, 0, 17], x["q"][30, 0, 17] = 1, -1
    return "dk", 0, 17


def _values_before(x):
    """dk_31 = -sum over earlier tokens of (dz_31 . u) k."""
    x["k"][0, 0, [0, 1]], x["k"][1, 0, [0, 1]], x["k"][31, 0, 2] = (1, 1), (-1, 1), 1
    x["v"][0, 0, [0, 1, 20]], x["v"][1, 0, [0, 1]], x["b"][:] = (1, A, E), (1, A), 1
    x["dl"][0, 0, 2, [0, 1, 20]] = 1, B, E
    return "dk", 31, 0


def _values_behind(x):
    """dk_0 = -sum over later tokens of (dz . u_0) k."""
    x["k"][0, 0, 0], x["k"][1, 0, [1, 2]], x["k"][31, 0, [1, 2]] = 1, (1, 1), (-1, 1)
    x["v"][0, 0, [0, 1, 20]], x["b"][:] = (1, A, E), 1
    x["dl"][0, 0, 2, [0, 1, 20]] = 1, B, E / 2
    x["dl"][0, 0, 1, 20] = E / 2
    return "dk", 0, 1


def _queries(x):
    """dq = h do, h in 24 bits."""
    x["st"][0, 0, 5, [3, 20]] = LONG, SHORT
    x["do"][9, 0, [3, 20]] = 1, -1
    return "dq", 9, 5


def _values(x):
    """dv_0 = sum over later tokens of (q . k_0) do, the factors in 24 bits."""
    x["k"][0, 0, [0, 1, 35]], x["b"][0] = (1, A, E), 1
    x["q"][3, 0, [0, 1, 35]], x["q"][31, 0, [0, 1]] = (1, B, E), (1, B)
    x["do"][3, 0, 9], x["do"][31, 0, 9] = 1, -1
    return "dv", 0, 9


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("case", [_behind, _replaced_back, _before, _errors, _values_seen, _values_before, _values_behind,
                                  _queries, _values], ids=lambda f: f.__name__[1:])
def test_gradients_of_whole_operands(case, dtype):
    x = _zeros(32)
    name, t, c = case(x)
    args = tuple(x[n] for n in ("q", "k", "v", "g", "b", "st"))
    at = ("dq", "dk", "dv").index(name)
    want = delta.delta_rule_backward(*args[:5], x["do"], [32], args[5], x["dl"])[at][t, 0, c]
    assert abs(want) in (2.0 ** -20, 2.0 ** -21)
    got = run(args, x["do"], [32], x["dl"], 1.0, dtype)[at]
    assert got[t, 0, c] == want


def _beyond(name, got, ref, terms, n):
    """got, in bf16, off by half a step of its own and by the fp32 roundings of `terms`, as delta_reference.check says."""
    size = np.maximum(np.abs(got), np.abs(ref))
    half = np.where(size > 0, 2.0 ** (np.floor(np.log2(np.maximum(size, 2.0 ** -126))) - 8), 0)
    over = np.maximum(np.abs(got - ref) - half, 0)
    tol = 2 * n * 2.0 ** -24 * terms + 1e-37
    norm, whole = np.linalg.norm(over), 2 * np.sqrt(n) * 2.0 ** -24 * np.linalg.norm(terms) + 1e-37
    print(f"[delta] {name}: beyond half a step / tolerance {np.max(over / tol):.3f}, of the norm {norm / whole:.3f}", flush=True)
    assert np.all(over <= tol) and norm <= whole, name


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c)).replace(" ", ""))
def test_outputs_show_their_own_rounding_alone(case):
    lens, G, H, K, V = case
    args = make(lens, G, H, K, V, "bf16", seed=len(lens) * K + V + 1)
    q, k, v, g, b, st = args
    scale = K ** -0.5
    o = _host(packed(args, lens, "bf16", scale)[0])
    terms, mass = delta.delta_rule_terms(q, k, v, g, b, lens, st, scale, 64)
    # what is in the state before a chunk has its own errors, in every direction
    over = scale * np.repeat(np.linalg.norm(q, axis=-1), H // G, 1)[..., None]
    per = np.concatenate([np.broadcast_to(mass[s], (n,) + mass.shape[1:]) for s, n in enumerate(lens)])
    _beyond("o", o, delta.delta_rule(q, k, v, g, b, lens, st, scale)[0], terms + over * np.maximum(per, terms), K + V + 64)


@pytest.mark.parametrize("case", GRADIENT_CASES, ids=lambda c: "-".join(map(str, c)).replace(" ", ""))
def test_gradients_show_their_own_rounding_alone(case):
    lens, G, H, K, V = case
    args = make(lens, G, H, K, V, "bf16", seed=len(lens) * K + V + 1)
    r = np.random.default_rng(K + 1)
    do = values(r.standard_normal(args[2].shape), "bf16")
    dl = r.standard_normal(args[5].shape).astype(np.float32)
    got = run(args, do, lens, dl, K ** -0.5, "bf16")
    ref = delta.delta_rule_backward(*args[:5], do, lens, args[5], dl, K ** -0.5)
    terms = gradient_terms(*args[:5], do, lens, args[5], dl, K ** -0.5, 64)
    for i, name in enumerate(("dq", "dk", "dv")):
        _beyond(name, got[i], ref[i], 2 * terms[i], K + V + 64)  # states' errors as large again

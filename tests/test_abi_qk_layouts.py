"""Which layouts of queries, keys and their outputs ss2d_qk_norm takes, on the CPU: all whose outputs lie apart and share
no address with the other side or, unless they are their own input, with that.  Addresses are fake; where a device exists
a valid call would launch kernels on them, and these tests are skipped."""
import random

import pytest

from test_abi_delta import norm, qk_sizes
from test_abi_tokens import ALIAS, NO_DEVICE, SHAPE, at, needs_no_device

D = 16


def _layouts(S, T, Hq, Hk):
    """name -> strides and offsets (elements) of queries and keys in one tensor."""
    H = max(Hq, Hk)
    row = (Hq + 2 * Hk) * D
    return {
        # rows of a projection, (S, T, ...) and (T, S, ...)
        "rows": ((T * row, row, D), 0, (T * row, row, D), Hq * D),
        "sequences inside": ((row, S * row, D), 0, (row, S * row, D), Hq * D),
        # q, k, v of a head side by side: (S, T, H, 3, D)
        "per head": ((T * H * 3 * D, H * 3 * D, 3 * D), 0, (T * H * 3 * D, H * 3 * D, 3 * D), D),
        # (S, 3, T, H, D)
        "planes": ((3 * T * H * D, H * D, D), 0, (3 * T * H * D, H * D, D), T * H * D),
        # heads before tokens: (S, Hq + 2 Hk, T, D)
        "heads first": ((T * row, D, T * D), 0, (T * row, D, T * D), Hq * T * D),
        # (S, T, D) of each head, a queries' head and a keys' head in turn
        "heads in turn": ((2 * H * T * D, D, 2 * T * D), 0, (2 * H * T * D, D, 2 * T * D), T * D),
    }


@needs_no_device
@pytest.mark.parametrize("S,T,Hq,Hk", [(2, 50, 4, 4), (1, 50, 4, 4), (3, 1, 4, 2), (1, 1, 2, 2), (2, 7, 4, 1), (2, 7, 1, 3)])
@pytest.mark.parametrize("name", sorted(_layouts(1, 1, 1, 1)))
def test_norms_over_their_inputs_in_one_tensor(name, S, T, Hq, Hk):
    sq, oq, sk, ok = _layouts(S, T, Hq, Hk)[name]
    for dtype, e in ((0, 4), (1, 2)):
        z = qk_sizes(S=S, T=T, Hq=Hq, Hk=Hk, q=sq, k=sk, qo=sq, ko=sk)
        q, k = at(1) + oq * e, at(1) + ok * e
        assert norm(z=z, dtype=dtype, q=q, k=k, qo=q, ko=k) == NO_DEVICE
        assert norm(z=z, dtype=dtype, q=q, k=k, qo=q, ko=k + e) == ALIAS
        assert norm(z=z, dtype=dtype, q=q, k=q, qo=q, ko=k) == ALIAS


def _addresses(start, n, stride):
    return {start + s * stride[0] + t * stride[1] + h * stride[2] + c
            for s in range(n[0]) for t in range(n[1]) for h in range(n[2]) for c in range(D)}


def _apart(n, stride):
    """Whether each axis of several steps over all that the narrower ones span."""
    span = D
    for s, m in sorted((s, m) for s, m in zip(stride, n) if m > 1):
        if s < span:
            return False
        span += (m - 1) * s
    return True


@needs_no_device
@pytest.mark.parametrize("seed", range(8))
def test_layouts_are_taken_if_and_only_if_they_share_no_address(seed):
    r = random.Random(seed)
    seen = {NO_DEVICE: 0, ALIAS: 0, SHAPE: 0}
    for _ in range(400):
        S, T, Hq, Hk = (r.choice([1, 2, 3]) for _ in range(4))
        Hk = r.choice([Hq, Hk])

        def strides():
            """Axes nested in some order with gaps now and then, one now and then too narrow."""
            out, span = [0, 0, 0], D
            for i in r.sample(range(3), 3):
                out[i] = span * r.choice([1, 1, 2, 3]) + r.choice([0, 0, 0, 5])
                span = out[i] * ((S, T, max(Hq, Hk))[i])
            if r.random() < 0.05:
                out[r.randrange(3)] //= 2
            return tuple(out)

        a, b = strides(), strides()
        which = {"q": (a, r.randrange(0, 20) * D), "k": (r.choice([a, a, b]), r.randrange(0, 60) * D)}
        for n, i in (("qo", "q"), ("ko", "k")):
            which[n] = which[i] if r.random() < 0.6 else (r.choice([a, b]), r.randrange(0, 120) * D + r.choice([0, 0, 3]))
        n = {x: (S, T, Hq if x[0] == "q" else Hk) for x in which}
        sets = {x: _addresses(o, n[x], s) for x, (s, o) in which.items()}

        def own(x):  # the output is its input
            return which[x][1] == which[x[0]][1] and all(
                m == 1 or p == q for m, p, q in zip(n[x], which[x][0], which[x[0]][0]))

        if not all(_apart(n[x], which[x][0]) for x in ("qo", "ko")):
            want = SHAPE
        elif sets["qo"] & sets["ko"] or any(sets[o] & sets[i] and not (o[0] == i and own(o))
                                            for o in ("qo", "ko") for i in "qk"):
            want = ALIAS
        else:
            want = NO_DEVICE
        got = norm(z=qk_sizes(S=S, T=T, Hq=Hq, Hk=Hk, **{x: s for x, (s, _) in which.items()}),
                   **{x: at(1) + 4 * o for x, (_, o) in which.items()})
        assert got == want, (S, T, Hq, Hk, which)
        seen[want] += 1
    assert all(seen.values())

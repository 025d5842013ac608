"""csa2_verify's drawn token where the mark lies close to a border between two tokens of a real softmax row, and on
rows of the largest vocabularies."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu


def _draw(target, probs, draft, u):
    """The token drawn for every row of u [batch, max_draft + 1] over the same rows target and probs."""
    import csa2_sparse_attention_decode_b200 as csa2
    B, k1 = u.shape
    dev = lambda x: torch.as_tensor(x, device="cuda")          # noqa: E731
    i32 = lambda x: dev(np.asarray(x, np.int32))               # noqa: E731
    acc, tok, err = i32(np.full(B, -9)), i32(np.full((B, k1), -9)), i32([0])
    csa2.csa2_verify(dev(target).expand(B, -1, -1).contiguous(),
                     None if probs is None else dev(probs).expand(B, -1, -1).contiguous(),
                     i32(np.full((B, k1 - 1), draft)), i32(np.full(B, k1 - 1)), dev(u), acc, tok, err)
    assert int(err) == 0 and not acc.any()
    return tok[:, 0].cpu().numpy()


def _row(r, V, kind):
    x = r.normal(size=V) * {"flat": 0.3, "usual": 3.0, "peaked": 3.0}[kind]
    if kind == "peaked":
        x[r.integers(0, V // 4)] = x.max() + 8                 # most of the mass in one token
    e = np.exp(x - x.max())
    return (e / e.sum()).astype(np.float32)


# fp64 sums of V weights are off by at most V * 2^-53 of the total, in whatever order, sums of groups of weights by
# 2^-42: under 2 * V * 2^-53 in all for the V here (2^-39.7 for 5000).  So are the mark and the border that it is
# compared with, and marks further than 4 * V * 2^-53 from any border have one answer.
@pytest.mark.parametrize("V", [131072, 100003, 5000])
@pytest.mark.parametrize("kind", ["flat", "usual", "peaked"])
@pytest.mark.parametrize("residual", ["none", "probs", "point"])
def test_marks_next_to_a_border(V, kind, residual):
    r = np.random.default_rng(V)
    target, probs, draft = _row(r, V, kind)[None, None], None, 0
    w = target[0, 0].astype(np.longdouble)
    if residual != "none":
        draft = int(r.integers(0, V))
        target = np.repeat(target, 2, 1)
        target[0, 0, draft] = 0                                # refused whatever u
        w = target[0, 0].astype(np.longdouble)
        if residual == "probs":
            probs = _row(r, V, kind)[None, None]
            probs[0, 0, draft] = max(probs[0, 0, draft], np.float32(1e-6))
            w = np.maximum(w - probs[0, 0].astype(np.longdouble), 0)
    c = np.cumsum(w)
    near = np.float32(c / c[-1])
    u = np.unique(np.concatenate([near, np.nextafter(near, np.float32(0)), np.nextafter(near, np.float32(2))]))
    u = u[(u >= 0) & (u < 1)]
    mark = u.astype(np.longdouble) * c[-1]
    at = np.searchsorted(c, mark, side="right")                # first index whose sum passes the mark
    gap = np.minimum(np.abs(c[np.minimum(at, V - 1)] - mark), np.abs(mark - c[np.maximum(at - 1, 0)])) / c[-1]
    fine = np.flatnonzero(gap > 4 * V * 2.0 ** -53)
    pick = fine[np.argsort(gap[fine])[:200]]
    want = at[pick]
    got = _draw(target, probs, draft, np.stack([np.full(len(pick), 0.5, np.float32)] * (target.shape[1] - 1) +
                                               [u[pick]], 1))
    off = np.flatnonzero(got != want)
    assert len(off) == 0, f"{len(off)} of {len(pick)} off, the first {float(gap[pick[off[0]]]):.2g} of the total from a border"


def test_weights_whose_sums_pass_the_range_of_fp32():
    V = 40000
    target = np.zeros((1, 1, V), np.float32)
    big = np.array([3, 4, 5, 19, 700, 20000, 20001, 39999])
    target[0, 0, big] = 2.0 ** 127             # finite each, not in fp32 together
    u = ((np.arange(8) + 0.5) / 8).astype(np.float32)
    assert _draw(target, None, 0, u[:, None]).tolist() == big.tolist()
    target[0, 0, big] = 2.0 ** -149            # the least there is
    assert _draw(target, None, 0, u[:, None]).tolist() == big.tolist()
    target = np.repeat(target, 2, 1)           # a refused draft, and what is left of p
    target[0, 0, big] = 2.0 ** 127
    probs = np.zeros((1, 1, V), np.float32)
    probs[0, 0, 9] = 1
    probs[0, 0, big] = 2.0 ** 126
    assert _draw(target, probs, 9, np.stack([np.full(8, 0.5, np.float32), u], 1)).tolist() == big.tolist()


@pytest.mark.parametrize("V", [7, 40000])
def test_an_infinite_weight_is_reported(V):
    import csa2_sparse_attention_decode_b200 as csa2
    i32 = lambda x: torch.as_tensor(np.asarray(x, np.int32), device="cuda")         # noqa: E731
    target = torch.full((3, 2, V), 1.0, device="cuda")
    target[1, 0, 5] = target[2, 1, 5] = float("inf")
    target[1, 0, 0] = 0                        # request 1 refuses its draft, request 2 keeps it
    probs = torch.full((3, 1, V), 0.5, device="cuda")
    acc, tok, err = i32([-9] * 3), i32([[-9] * 2] * 3), i32([0])
    csa2.csa2_verify(target, probs, i32([[0]] * 3), i32([1] * 3), torch.full((3, 2), 0.25, device="cuda"), acc, tok, err)
    assert int(err) == 4 and acc.tolist() == [1, 0, 1]
    assert tok.tolist() == [[0, V // 4], [V - 1, -1], [0, V - 1]]

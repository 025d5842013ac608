"""The calls around the layers against plain 64-bit computations: draft
verification, the token plan, and the head norm with rotation."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

U24, U8 = 2.0 ** -24, 2.0 ** -8                # half steps of f32 and bf16, relative


def _csa2():
    import csa2_sparse_attention_decode_b200 as csa2
    return csa2


def _i32(x):
    return torch.as_tensor(np.asarray(x, np.int32), device="cuda")


# ---------------------------------------------------------------- verification
def _verify(target, probs, draft, n_draft, u):
    csa2 = _csa2()
    B, k1, _ = target.shape
    acc, tok, err = _i32(np.full(B, -9)), _i32(np.full((B, k1), -9)), _i32([0])
    csa2.csa2_verify(torch.as_tensor(target, device="cuda"),
                     None if probs is None else torch.as_tensor(probs, device="cuda"), _i32(draft), _i32(n_draft),
                     torch.as_tensor(np.asarray(u, np.float32), device="cuda"), acc, tok, err)
    return acc.cpu().numpy(), tok.cpu().numpy(), int(err)


def _verify_ref(target, probs, draft, n_draft, u):
    """Outcome per request; a drawn index is given with the cumulative weights, to judge rounding at a border."""
    B, k1, V = target.shape
    res = []
    for b in range(B):
        n = 0
        while n < n_draft[b] and 0 <= draft[b][n] < V and \
                np.float64(u[b][n]) * (1.0 if probs is None else np.float64(probs[b, n, draft[b][n]])) < \
                np.float64(target[b, n, draft[b][n]]):
            n += 1
        w = np.maximum(np.nan_to_num(target[b, n].astype(np.float64)), 0)
        if n < n_draft[b]:
            q = np.eye(1, V, draft[b][n] if 0 <= draft[b][n] < V else V)[0] if probs is None else \
                probs[b, n].astype(np.float64)
            r = np.maximum(w - q, 0)
            w = r if r.sum() > 0 else w
        c = np.cumsum(w)
        res.append((n, int(np.argmax(c > np.float64(u[b][k1 - 1]) * c[-1]))))
    return res


def _check_verify(target, probs, draft, n_draft, u):
    acc, tok, err = _verify(target, probs, draft, n_draft, u)
    for b, (n, x) in enumerate(_verify_ref(target, probs, draft, n_draft, u)):
        want = [int(d) for d in draft[b][:n]] + [x] + [-1] * (target.shape[1] - 1 - n)
        assert acc[b] == n and tok[b].tolist() == want, (b, acc[b], tok[b], n, want)
    return err


@pytest.mark.parametrize("batch,k,vocab", [(1, 0, 1), (3, 1, 33), (5, 3, 1000), (64, 2, 16383), (7, 31, 16384),
                                           (4, 5, 131072), (2, 1, 100003)])
@pytest.mark.parametrize("with_probs", [True, False])
def test_verify_random(batch, k, vocab, with_probs):
    r = np.random.default_rng(batch * 100 + k)
    # dyadic weights: every sum is exact in 64 bits, so no border moves by rounding
    target = np.round(r.random((batch, k + 1, vocab)) ** 4 * 4096).astype(np.float32) / 4096
    target[..., 0] += 1 / 4096                 # no row without weight
    probs = np.round(r.random((batch, k, vocab)) ** 4 * 4096).astype(np.float32) / 4096 if with_probs else None
    draft = r.integers(0, vocab, (batch, k))
    n_draft = r.integers(0, k + 1, batch)
    u = np.round(r.random((batch, k + 1)) * 1024 * 0.999).astype(np.float32) / 1024
    u[:, :k] *= 0.25                           # some runs of accepted drafts
    assert _check_verify(target, probs, draft, n_draft, u) == 0


def test_verify_borders_and_point_masses():
    V = 40000
    target = np.zeros((6, 2, V), np.float32)
    probs = np.zeros((6, 1, V), np.float32)
    draft = np.full((6, 1), 7)
    target[:, :, [5, 17, 39999]] = [0.25, 0.5, 0.25]
    target[0, 0, 7] = probs[0, 0, 7] = 1.0     # equal: kept for every u below one
    probs[1, 0, 7] = 0.5                       # target zero there: refused even at u = 0
    probs[2, 0] = 2 * target[2, 0]             # nothing is left of p: drawn from p itself
    probs[2, 0, 7] = 1.0
    target[3, 1] = 0
    target[3, 1, 123] = 3.0                    # one token, not normalised
    target[3, 0, 7] = 1.0
    probs[3, 0, 7] = 0.5
    target[4, 0, 7], probs[4, 0, 7] = 0.25, 0.5
    target[5, 0, 7], probs[5, 0, 7] = 0.25, 0.5
    for last in (0.0, 0.25, 0.75, 1 - 2.0 ** -24):
        u = np.array([[1 - 2.0 ** -24, last], [0, last], [0.1, last], [0.9, last], [0.5, last],
                      [0.5 - 2.0 ** -20, last]], np.float32)
        assert _check_verify(target, probs, draft, np.ones(6, int), u) == 0


def test_verify_bad_data_is_reported_not_followed():
    V = 20000
    target = np.full((4, 3, V), 1 / 4096, np.float32)
    draft = np.array([[V, 3], [-1, 3], [2, 3], [2, 3]])
    u = np.full((4, 3), 0.5, np.float32)
    u[:, :2] = 0
    assert _check_verify(target, None, draft, [2, 2, 2, 2], u) == 3      # token outside the vocabulary
    acc, tok, err = _verify(target, None, draft * 0 + 1, [3, -1, 2, 0], u)
    assert err == 4 and acc.tolist() == [2, 0, 2, 0]                     # counts clamped to 0..2
    target[2] = 0
    target[3] = np.nan
    acc, tok, err = _verify(target, None, draft * 0 + 1, [2, 2, 2, 2], u)
    assert err == 4 and acc.tolist() == [2, 2, 0, 0] and tok[2].tolist() == [V - 1, -1, -1] == tok[3].tolist()
    target[3, :, 9] = 0.5                      # NaN elsewhere is never drawn
    acc, tok, err = _verify(target[3:], None, draft[3:] * 0 + 1, [2], u[3:])
    assert err == 0 and tok[0].tolist() == [9, -1, -1]


# ---------------------------------------------------------------- token plan
def _plan_state(r, B, past_hi, new_lo, new_hi, drop, spare=7, room=None):
    past = r.integers(0, past_hi + 1, B)
    m = 1 + (r.random(B) < 0.4).astype(int)
    new = r.integers(new_lo, new_hi + 1, B)
    new = np.where(r.random(B) < drop, -r.integers(0, past + 1), new)
    own = -(-(past // m) // 64)
    width = int((-(-(past + np.maximum(new, 0)) // 64)).max()) + 1
    total = int(np.maximum(own, -(-((past + new) // m) // 64)).sum()) + spare
    perm = r.permutation(total).astype(np.int32)
    table = np.full((B, width), -5, np.int32)
    at = 0
    for b in range(B):
        table[b, :own[b]] = perm[at:at + own[b]]
        at += own[b]
    free = np.full(total, -6, np.int32)
    free[:total - at] = perm[at:]
    return {"past": past, "new": new, "m": m, "table": table, "free": free, "n_free": total - at,
            "room": int(np.maximum(new, 0).sum()) + 3 if room is None else room}


def _plan(s, table=None, free=None):
    csa2 = _csa2()
    B = len(s["past"])
    o = {"table": _i32(s["table"]), "free": _i32(s["free"]), "n_free_out": _i32([-1]), "cu": _i32(np.zeros(B + 1)),
         "req": _i32(np.full(s["room"], -7)), "pos": _i32(np.full(s["room"], -7)),
         "slot": _i32(np.full(s["room"], -7)), "err": _i32([0])}
    args = (_i32(s["past"]), _i32(s["new"]), _i32(s["m"]), o["table"], o["free"], _i32([s["n_free"]]),
            o["n_free_out"], o["cu"], o["req"], o["pos"], o["slot"], o["err"])
    csa2.csa2_plan_tokens(*args)
    once = {k: v.cpu().numpy().copy() for k, v in o.items()}
    csa2.csa2_plan_tokens(*args)               # repeated before anything changes: the same again
    for k, v in o.items():
        assert np.array_equal(once[k], v.cpu().numpy()), k
    return once


def _plan_ref(s):
    """Request by request, as an allocator would."""
    table, stack, n_pages = s["table"].copy(), list(s["free"][:s["n_free"]]), len(s["free"])
    err = 0
    B = len(s["past"])
    pages = lambda t, m: -(-(t // m) // 64)    # noqa: E731
    new = list(s["new"])
    for b in range(B):
        past, m = s["past"][b], s["m"][b]
        if m not in (1, 2) or past < 0 or past > table.shape[1] * 64 * m or past + new[b] < 0:
            err, new[b] = err or 4, None
        elif past + new[b] > table.shape[1] * 64 * m:
            err, new[b] = err or 2, 0
    for b in range(B):
        if new[b] is not None:
            stack += list(table[b, pages(s["past"][b] + new[b], s["m"][b]):pages(s["past"][b], s["m"][b])])
    full = np.array(s["free"])
    full[s["n_free"]:len(stack)] = stack[s["n_free"]:]
    cu, req, pos, slot, no_rows, no_pages, rows = [0], [], [], [], False, False, 0
    for b in range(B):
        n = new[b]
        if n is not None and n > 0:
            m, past = s["m"][b], s["past"][b]
            rows += n
            get = pages(past + n, m) - pages(past, m)
            if rows > s["room"]:
                err, n = err or 2, 0
            elif get > 0 and (no_pages or get > len(stack)):
                err, n, no_pages = err or 2, 0, True
            else:
                for j in range(get):
                    table[b, pages(past, m) + j] = stack.pop()
            for t in range(past, past + n):
                e = t // m
                req.append(b)
                pos.append(t)
                slot.append(-1 if m == 2 and t % 2 == 0 else table[b, e // 64] * 64 + e % 64)
        cu.append(cu[-1] + max(0, n or 0))
    return {"table": table, "free": full, "n_free_out": np.array([len(stack)]), "cu": np.array(cu), "req": req,
            "pos": pos, "slot": slot, "err": np.array([err])}


def _check_plan(s):
    got, want = _plan(s), _plan_ref(s)
    n = len(want["req"])
    for k in ("table", "free", "n_free_out", "cu", "err"):
        assert np.array_equal(got[k], want[k]), k
    for k in ("req", "pos", "slot"):
        assert got[k][:n].tolist() == list(want[k]), k
        assert (got[k][n:] == -7).all(), k     # rows behind the last token stay
    return got


@pytest.mark.parametrize("B,past_hi,new_lo,new_hi,drop", [
    (1, 0, 0, 0, 0), (1, 200, 1, 1, 0), (3, 130, 0, 3, 0.5), (64, 5000, 1, 1, 0), (255, 700, 0, 2, 0.3),
    (256, 70, 1, 5, 0.1), (257, 300, 0, 200, 0.5), (4096, 66, 0, 2, 0.4), (5, 0, 1, 20000, 0), (9, 30000, 0, 9000, 0.4)])
def test_plan_against_an_allocator(B, past_hi, new_lo, new_hi, drop):
    got = _check_plan(_plan_state(np.random.default_rng(B + new_hi), B, past_hi, new_lo, new_hi, drop))
    assert got["err"][0] == 0


def test_plan_grants_no_page_twice():
    s = _plan_state(np.random.default_rng(5), 40, 4000, 1, 3000, 0.3)
    got = _plan(s)
    after = s["past"] + np.where(s["new"] < 0, s["new"], np.diff(got["cu"]))
    held = np.concatenate([got["table"][b, :-(-(after[b] // s["m"][b]) // 64)] for b in range(40)] +
                          [got["free"][:got["n_free_out"][0]]])
    assert sorted(held.tolist()) == list(range(len(s["free"])))


@pytest.mark.parametrize("short", ["pages", "rows", "both"])
def test_plan_serves_in_order_while_pages_and_rows_last(short):
    r = np.random.default_rng(11)
    s = _plan_state(r, 30, 500, 0, 300, 0.1, spare=0)
    if short != "rows":
        s["free"][s["n_free"] // 2:] = -6
        s["n_free"] //= 2
    if short != "pages":
        s["room"] //= 2
    got = _check_plan(s)
    assert got["err"][0] == 2


def test_plan_bad_lengths_and_pages_are_reported_not_followed():
    r = np.random.default_rng(3)
    s = _plan_state(r, 12, 300, 1, 100, 0)
    cap = s["table"].shape[1] * 64
    s["m"][1], s["past"][2], s["new"][3], s["past"][4] = 3, -1, -s["past"][3] - 1, 2 * cap + 1
    assert _check_plan(s)["err"][0] == 4
    s = _plan_state(r, 6, 300, 1, 100, 0)
    s["new"][2] = 2 * s["table"].shape[1] * 64 + 1
    s["room"] += 200
    assert _check_plan(s)["err"][0] == 2
    # page ids outside the pool, owned and free
    s = _plan_state(r, 4, 300, 100, 200, 0)
    s["m"][:], s["past"][:] = 1, 100
    s["table"][:, :2] = np.arange(8).reshape(4, 2)
    s["table"][1, 1] = len(s["free"])
    s["free"][:] = np.arange(len(s["free"]))
    s["n_free"] = len(s["free"])
    s["free"][-1] = -3
    got = _plan(s)
    assert got["err"][0] == 1
    a, b = got["cu"][1], got["cu"][2]
    assert (got["slot"][a:b][:28] == -1).all() and (got["slot"][:28] >= 0).all()
    assert got["table"][0, 2] == -1 and (got["slot"][28:a][:64] == -1).all()


# ---------------------------------------------------------------- norm with rotation
def _norm_ref(x, w, pos, freq, halves, eps, norm=True, inverse=False):
    """fp64 result and, per element, the magnitude its rounding errors scale with."""
    y = x.double()
    if norm:
        y = y / torch.sqrt((y * y).mean(-1, keepdim=True) + float(np.float32(eps))) * w.double()
    mag = y.abs()
    if freq is None:
        return y, mag
    R = 2 * freq.numel()
    t = pos.double()[:, None, None] * freq.double() * (-1 if inverse else 1)
    c, s = torch.cos(t), torch.sin(t)
    tail = y[..., -R:].clone()
    a, b = (tail[..., :R // 2], tail[..., R // 2:]) if halves else (tail[..., 0::2], tail[..., 1::2])
    ra, rb, m = a * c - b * s, a * s + b * c, a.abs() + b.abs()
    y, mag = y.clone(), mag.clone()
    y[..., -R:] = torch.cat([ra, rb], -1) if halves else torch.stack([ra, rb], -1).flatten(-2)
    mag[..., -R:] = torch.cat([m, m], -1) if halves else torch.stack([m, m], -1).flatten(-2)
    return y, mag


# The fp32 part: a sum of up to 512 squares in runs of 16 and a tree of 5 (21
# roundings, halved by the root), the root (2 ulp), two products, the turn's
# rounding (2 pi * 2^-25 rad), sine and cosine (2 ulp), a product and a sum:
# under 32 half steps of the pair's magnitude.
def _check_norm(got, ref, mag, what):
    half = U8 if got.dtype == torch.bfloat16 else U24
    tol = half * ref.abs() + 32 * U24 * mag * (1 + half) + 1e-38
    bad = (got.double() - ref).abs() > tol
    assert not bad.any(), f"{what}: {int(bad.sum())} off, first {bad.nonzero()[0].tolist()}"


def _freq(R):
    return (10000.0 ** (-torch.arange(0, R, 2, dtype=torch.float64) / R)).float().cuda() if R else None


@pytest.mark.parametrize("dim", [64, 128, 256, 512])
@pytest.mark.parametrize("n,heads,kv,pad,rot_of", [(1, 64, 1, 0, 8), (1, 1, 0, 0, 1), (3, 0, 1, 8, 2), (17, 5, 2, 24, 1),
                                                   (300, 32, 1, 0, 4), (1200, 3, 1, 128, 1), (40, 128, 3, 0, 0)])
@pytest.mark.parametrize("halves", [False, True])
def test_norm_rope(dim, n, heads, kv, pad, rot_of, halves):
    csa2 = _csa2()
    g = torch.Generator(device="cuda").manual_seed(dim + n)
    rot = max(16, dim // rot_of) if rot_of else 0
    wide = (heads + kv) * dim + pad
    x = (torch.randn(n, wide, generator=g, device="cuda") *
         torch.exp(2 * torch.randn(n, 1, generator=g, device="cuda"))).to(torch.bfloat16)
    q = x[:, :heads * dim].view(n, heads, dim) if heads else None
    k = x[:, heads * dim:(heads + kv) * dim].view(n, kv, dim) if kv else None
    pos = torch.randint(-5, 2 ** 31 - 1, (n,), generator=g, device="cuda", dtype=torch.int32)
    pos[0] = 0
    wq, wk = (torch.randn(dim, generator=g, device="cuda") for _ in range(2))
    freq = _freq(rot)
    qo = torch.empty(n, heads, dim, dtype=torch.bfloat16, device="cuda") if heads else None
    ko = torch.empty(n, kv, dim, dtype=torch.bfloat16, device="cuda") if kv else None
    kf = torch.empty(n, kv, dim, device="cuda") if kv else None
    flags = csa2.ROPE_HALVES if halves else 0
    csa2.csa2_norm_rope(q, k, pos, freq, wq if heads else None, wk if kv else None, 1e-6, qo, ko, kf, flags=flags)
    if heads:
        _check_norm(qo, *_norm_ref(q, wq, pos, freq, halves, 1e-6), "q")
    if kv:
        ref = _norm_ref(k, wk, pos, freq, halves, 1e-6)
        _check_norm(ko, *ref, "k bf16")
        _check_norm(kf, *ref, "k f32")
        only = torch.empty_like(kf)
        csa2.csa2_norm_rope(None, k, pos, freq, None, wk, 1e-6, None, None, only, flags=flags)
        assert torch.equal(only, kf)


@pytest.mark.parametrize("halves", [False, True])
def test_norm_rope_in_place_padded_and_back(halves):
    csa2 = _csa2()
    g = torch.Generator(device="cuda").manual_seed(7)
    n, H, d, keep = 33, 6, 512, 21
    flags = csa2.ROPE_HALVES if halves else 0
    x = torch.randn(n, H, d, generator=g, device="cuda").to(torch.bfloat16)
    pos = torch.randint(0, 1 << 20, (n,), generator=g, device="cuda", dtype=torch.int32)
    freq = _freq(64)
    y = x.clone()
    csa2.csa2_norm_rope(y, None, pos, freq, None, None, 0.0, y, None, n_valid=_i32([keep]),
                        flags=flags | csa2.ROPE_NO_NORM)
    assert torch.equal(y[keep:], x[keep:])     # padding: neither read nor written
    _check_norm(y[:keep], *[v[:keep] for v in _norm_ref(x, None, pos, freq, halves, 0, norm=False)], "in place")
    back = torch.empty_like(y)
    csa2.csa2_norm_rope(y, None, pos, freq, None, None, 0.0, back, None,
                        flags=flags | csa2.ROPE_NO_NORM | csa2.ROPE_INVERSE)
    _check_norm(back, *_norm_ref(y, None, pos, freq, halves, 0, norm=False, inverse=True), "inverse")
    for bad in (-4, 0):
        z = x.clone()
        csa2.csa2_norm_rope(z, None, pos, freq, None, None, 0.0, z, None, n_valid=_i32([bad]), flags=csa2.ROPE_NO_NORM)
        assert torch.equal(z, x)


def test_norm_rope_zero_rows_and_nan_stay_in_their_row():
    csa2 = _csa2()
    x = torch.randn(4, 3, 128, device="cuda").to(torch.bfloat16)
    x[1, 1] = 0
    x[2, 0, 5] = float("nan")
    w = torch.ones(128, device="cuda")
    pos = _i32([0, 1, 2, 3])
    out = torch.empty_like(x)
    csa2.csa2_norm_rope(x, None, pos, _freq(128), w, None, 1e-6, out, None)
    assert (out[1, 1] == 0).all() and out[2, 0].isnan().all()
    clean = torch.ones(4, 3, dtype=torch.bool, device="cuda")
    clean[2, 0] = False
    assert out[clean].isfinite().all()

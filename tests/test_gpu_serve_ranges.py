"""The calls around the layers at the far ends of what they take: vocabularies up to 2^28, 1024 heads, and prompt
attention over more row tiles than several SMs may share."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu


def _csa2():
    import csa2_sparse_attention_decode_b200 as csa2
    return csa2


@pytest.mark.parametrize("V", [2200003, 5000000])
@pytest.mark.parametrize("kind", ["usual", "peaked"])
def test_verify_rows_of_millions(V, kind):
    # several blocks of weights a lane, and a search of several rounds
    from test_gpu_verify_sums import _draw, _row
    r = np.random.default_rng(V)
    target = np.repeat(_row(r, V, kind)[None, None], 2, 1)
    draft = int(r.integers(0, V))
    target[0, 0, draft] = 0
    probs = _row(r, V, "flat")[None, None]
    u = r.random(6).astype(np.float32)
    for q in (None, probs):
        w = target[0, 0].astype(np.longdouble)
        w = w if q is None else np.maximum(w - q[0, 0].astype(np.longdouble), 0)
        c = np.cumsum(w)
        mark = u.astype(np.longdouble) * c[-1]
        at = np.searchsorted(c, mark, side="right")
        gap = np.minimum(c[at] - mark, mark - c[np.maximum(at - 1, 0)]) / c[-1]
        fine = gap > 4 * V * 2.0 ** -53        # as in the test of marks next to a border
        assert fine.sum() >= 3
        got = _draw(target, q, draft, np.stack([np.full(6, 0.5, np.float32), u], 1))
        assert got[fine].tolist() == at[fine].tolist()


@pytest.mark.slow
def test_verify_the_largest_vocabulary():
    csa2 = _csa2()
    V, B, step = 1 << 28, 5, 1024
    target = torch.zeros(B, 1, V, device="cuda")
    target[:, :, 7::step] = 1                  # 2^18 weights: every mark below lies in the middle of one
    k = [0, 1, 77777, (1 << 18) - 2, (1 << 18) - 1]
    u = torch.tensor([[(x + 0.5) / (1 << 18)] for x in k], device="cuda")
    i32 = dict(dtype=torch.int32, device="cuda")
    acc, tok, err = torch.full((B,), -9, **i32), torch.full((B, 1), -9, **i32), torch.zeros(1, **i32)
    csa2.csa2_verify(target, None, torch.zeros(B, 0, **i32), torch.zeros(B, **i32), u, acc, tok, err)
    assert int(err) == 0 and acc.tolist() == [0] * B and tok[:, 0].tolist() == [7 + step * x for x in k]


@pytest.mark.parametrize("dim", [64, 512])
@pytest.mark.parametrize("heads,kv", [(1024, 1024), (1023, 0), (0, 1021), (1, 1024)])
@pytest.mark.parametrize("halves", [False, True])
def test_norm_of_a_thousand_heads(dim, heads, kv, halves):
    from test_gpu_serve import _check_norm, _freq, _norm_ref
    csa2 = _csa2()
    g = torch.Generator(device="cuda").manual_seed(heads + kv + dim)
    n = 5
    x = torch.randn(n, heads + kv, dim, generator=g, device="cuda").to(torch.bfloat16)
    q, k = (x[:, :heads] if heads else None), (x[:, heads:] if kv else None)
    pos = torch.randint(0, 1 << 20, (n,), generator=g, device="cuda", dtype=torch.int32)
    w, freq = torch.randn(dim, generator=g, device="cuda"), _freq(32)
    qo = torch.empty(n, heads, dim, dtype=torch.bfloat16, device="cuda") if heads else None
    ko, kf = (torch.empty(n, kv, dim, dtype=t, device="cuda") if kv else None for t in (torch.bfloat16, torch.float32))
    csa2.csa2_norm_rope(q, k, pos, freq, w if heads else None, w if kv else None, 1e-6, qo, ko, kf,
                        flags=csa2.ROPE_HALVES if halves else 0)
    for got, src in ((qo, q), (ko, k), (kf, k)):
        if got is not None:
            _check_norm(got, *_norm_ref(src, w, pos, freq, halves, 1e-6), "heads")


@pytest.mark.parametrize("f32", [False, True])
def test_whole_row_tiles_whose_tokens_straddle_them(f32):
    # 20 heads: 64-row tiles begin and end inside tokens; over 896 tiles, no window, several requests
    from test_gpu_prompt import _check_all
    _check_all([1500, 1, 0, 1399], [0, 700, 3, 200], 20, 0, f32, seed=20, extra_q=7)


@pytest.mark.parametrize("heads", [64, 65])
def test_decode_tokens_past_the_shared_row_tiles(heads):
    # more single tokens than the split path plans, with pasts from nothing to many key tiles
    from test_gpu_prompt import _check_all
    n = 1000
    past = [(i * 37) % 300 for i in range(n)]
    past[n // 3], past[-1] = 5000, 3000
    _check_all([1] * n, past, heads, 0, False, seed=heads)


def test_verify_the_largest_batch():
    csa2 = _csa2()
    B, V = 65535, 33
    g = torch.Generator(device="cuda").manual_seed(1)
    i32 = dict(dtype=torch.int32, device="cuda")
    target = torch.randint(0, 64, (B, 2, V), generator=g, device="cuda").float()       # exact sums
    target[..., 0] += 1
    draft = torch.randint(0, V, (B, 1), generator=g, **i32)
    u = torch.randint(0, 256, (B, 2), generator=g, device="cuda") / 256
    n_draft = torch.randint(0, 2, (B,), generator=g, **i32)
    acc, tok, err = torch.empty(B, **i32), torch.empty(B, 2, **i32), torch.zeros(1, **i32)
    csa2.csa2_verify(target, None, draft, n_draft, u, acc, tok, err)
    p = target.double()
    kept = (n_draft == 1) & (u[:, 0].double() < p[:, 0].gather(1, draft.long())[:, 0])
    w = torch.where(kept[:, None], p[:, 1], p[:, 0])
    rest = (w - torch.zeros_like(w).scatter(1, draft.long(), 1.0)).clamp_min(0)
    refused = (n_draft == 1) & ~kept
    w = torch.where(refused[:, None] & (rest.sum(1, keepdim=True) > 0), rest, w)
    c = w.cumsum(1)
    x = (c > u[:, 1:].double() * c[:, -1:]).int().argmax(1)
    assert int(err) == 0 and torch.equal(acc, kept.int())
    assert torch.equal(tok.gather(1, kept.long()[:, None])[:, 0].long(), x)
    assert torch.equal(tok[kept][:, 0], draft[kept][:, 0]) and (tok[~kept][:, 1] == -1).all()


@pytest.mark.parametrize("dim,halves", [(64, True), (64, False), (256, True)])
def test_norm_of_more_tokens_than_warps(dim, halves):
    from test_gpu_serve import _check_norm, _freq, _norm_ref
    csa2 = _csa2()
    g = torch.Generator(device="cuda").manual_seed(dim)
    n, live = 100001, 99990
    x = torch.randn(n, 2, dim, generator=g, device="cuda").to(torch.bfloat16)
    pos = torch.randint(0, 1 << 20, (n,), generator=g, device="cuda", dtype=torch.int32)
    w, freq = torch.randn(dim, generator=g, device="cuda"), _freq(32)
    out = torch.full_like(x, 7.0)
    csa2.csa2_norm_rope(x[:, :2], None, pos, freq, w, None, 1e-6, out, None,
                        n_valid=torch.tensor([live], dtype=torch.int32, device="cuda"),
                        flags=csa2.ROPE_HALVES if halves else 0)
    _check_norm(out[:live], *(y[:live] for y in _norm_ref(x, w, pos, freq, halves, 1e-6)), "tokens")
    assert (out[live:] == 7).all()


@pytest.mark.parametrize("heads,window", [(8, 0), (64, 128), (8, 50)])
def test_thousands_of_requests_most_of_them_empty(heads, window):
    from test_gpu_prompt import _check_all
    n = 5000
    new = [1 if i % 11 == 0 else 3 if i % 501 == 5 else 0 for i in range(n)]
    past = [(i * 13) % 40 if i % 2 else 0 for i in range(n)]
    _check_all(new, past, heads, window, False, seed=heads, extra_q=3)


@pytest.mark.parametrize("f32", [False, True])
def test_latents_inside_a_wider_row(f32):
    # rows that begin 16 bytes into a projection's, the first of them not its first
    from test_gpu_prompt import _call, _check, _cu, _inputs, _ref
    for heads, window, new, kv in ((64, 128, 300, 300), (16, 0, 20, 700), (64, 0, 2, 9000)):
        q, lat = _inputs(heads, [new], [kv], heads)
        wide = torch.full((kv + 2, 584), 3.0, dtype=torch.bfloat16, device="cuda")
        wide[1:kv + 1, 8:520] = lat
        out, lse, err = _call(q, wide[1:kv + 1, 8:520], _cu([new]), _cu([kv]), window, f32)
        same, same_lse, _ = _call(q, lat.contiguous(), _cu([new]), _cu([kv]), window, f32)
        assert int(err) == 0 and torch.equal(out, same) and torch.equal(lse, same_lse)
        lo = max(0, kv - window) if window else 0
        _check(out[-1:], lse[-1:], _ref(q[-1:], lat[lo:], kv - 1 - lo, 0))

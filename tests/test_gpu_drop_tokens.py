"""Tokens that were written to a cache and are dropped again: csa2_plan_tokens takes their pages back, and
csa2_prefill over the window's tokens takes their traces out of the ring, the pending pair and the last summary."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

M = [1, 2, 1, 2, 1, 2]
KEPT = [190, 129, 62, 255, 3, 128]             # tokens that stay
N_PAGES = 32


def _i32(x):
    return torch.as_tensor(x, dtype=torch.int32, device="cuda")


def _cache(csa2):
    table = torch.full((len(M), 8), -1, dtype=torch.int32, device="cuda")
    cache = csa2.Cache(table, N_PAGES, M)
    cache.pool.zero_()
    return cache, {"free": _i32(range(N_PAGES)), "n_free": _i32([N_PAGES])}


def _plan(csa2, cache, s, n_new):
    rows = [_i32([0] * 2000) for _ in range(3)]
    out = _i32([0])
    csa2.csa2_plan_tokens(cache.n_tokens, _i32(n_new), cache.m, cache.page_table, s["free"], s["n_free"], out,
                          _i32([0] * (len(M) + 1)), *rows, cache.error)
    s["n_free"] = out


def _append(csa2, cache, tokens, at, count):
    """Tokens at[b] .. at[b] + count[b] - 1 (at most 2 each) of every request."""
    pick = [x.new_zeros(len(M), 2, *x.shape[2:]) for x in tokens]
    for b in range(len(M)):
        for p, x in zip(pick, tokens):
            p[b, :count[b]] = x[b, at[b]:at[b] + count[b]]
    csa2.csa2_append(cache, *pick, _i32(count))


def _prefill(csa2, cache, tokens, b, begin, end):
    csa2.csa2_prefill(cache, b, begin, end, *(x[b, begin:end].contiguous() for x in tokens))


def _state(cache, n):
    """What the calls read of every request with n[b] tokens."""
    got = []
    planes = [(0, 256, 64), (N_PAGES * 16384, 32, 64), (N_PAGES * 18432, 128, 64), (N_PAGES * 26624, 128, 8)]
    for b, m in enumerate(M):
        entries = n[b] // m
        for off, width, rows in planes:
            plane = cache.pool[off:off + N_PAGES * rows * width].view(-1, width)
            k = torch.arange(entries if rows == 64 else -(-entries // 8), device="cuda")
            got.append(plane[cache.page_table[b].long()[k // rows] * rows + k % rows])
        ring = cache.swa.view(len(M), 66048)[b]
        pos = torch.arange(max(0, n[b] - 128), n[b], device="cuda") % 128
        got.append(ring[:65536].view(128, 512)[pos])
        got.append(ring[65536:].view(torch.float32)[pos])
        if m == 2 and n[b] % 2:
            got.append(cache.pending.view(len(M), -1)[b, :641])
    return [x.clone() for x in got] + [cache.n_tokens.clone()]


@pytest.mark.parametrize("dropped", [[1, 1, 1, 1, 1, 1], [4, 3, 2, 4, 3, 2], [2, 4, 4, 1, 4, 4]])
def test_dropped_tokens_leave_no_trace(dropped):
    import csa2_sparse_attention_decode_b200 as csa2
    g = torch.Generator(device="cuda").manual_seed(sum(dropped))
    B, most = len(M), max(KEPT) + 16
    tokens = (torch.randn(B, most, 512, generator=g, device="cuda"), torch.randn(B, most, 128, generator=g, device="cuda"),
              torch.randn(B, most, generator=g, device="cuda"))
    plain, s_plain = _cache(csa2)
    other, s_other = _cache(csa2)
    _plan(csa2, plain, s_plain, KEPT)
    _plan(csa2, other, s_other, KEPT)
    for b in range(B):
        _prefill(csa2, plain, tokens, b, 0, KEPT[b])
        _prefill(csa2, other, tokens, b, 0, KEPT[b])
    # tokens that will not stay, two at a time
    at = list(KEPT)
    for _ in range(2):
        count = [max(0, min(2, KEPT[b] + dropped[b] - at[b])) for b in range(B)]
        _plan(csa2, other, s_other, count)
        wrong = tuple(x.flip(1).contiguous() for x in tokens)
        _append(csa2, other, wrong, at, count)
        at = [a + c for a, c in zip(at, count)]
    assert other.n_tokens.tolist() == at == [k + d for k, d in zip(KEPT, dropped)]
    _plan(csa2, other, s_other, [-d for d in dropped])
    assert int(s_other["n_free"]) == int(s_plain["n_free"])
    assert not all(torch.equal(x, y) for x, y in zip(_state(plain, KEPT), _state(other, KEPT)))
    for b in range(B):
        begin = max(0, KEPT[b] - 128) // M[b] * M[b]
        _prefill(csa2, other, tokens, b, begin, KEPT[b])
    n = list(KEPT)
    for step in range(3):                      # as it is, and after tokens that come next
        for x, y in zip(_state(plain, n), _state(other, n)):
            assert torch.equal(x, y)
        q = torch.randn(B, 16, 512, generator=g, device="cuda").to(torch.bfloat16)
        ix = torch.randn(B, 32, 128, generator=g, device="cuda").to(torch.bfloat16)
        hw = torch.rand(B, 32, generator=g, device="cuda")
        seen = []
        for cache in (plain, other):
            topk, out = torch.empty(B, 512, dtype=torch.int32, device="cuda"), torch.empty(B, 16, 512, device="cuda")
            ws = csa2.workspace(cache)
            csa2.csa2_index(cache, csa2.INDEX_FLAT, ix, hw, None, None, topk, ws)
            csa2.csa2_attend(cache, q, topk, 1 / math.sqrt(512), out, ws)
            seen.append((topk, out))
        assert torch.equal(seen[0][0], seen[1][0]) and torch.equal(seen[0][1], seen[1][1])
        count = [1 + (b + step) % 2 for b in range(B)]
        for cache, s in ((plain, s_plain), (other, s_other)):
            _plan(csa2, cache, s, count)
            _append(csa2, cache, tokens, n, count)
        n = [a + c for a, c in zip(n, count)]
    assert csa2.csa2_get_device_error(plain) == 0 == csa2.csa2_get_device_error(other)

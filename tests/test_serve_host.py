"""Refusals of the calls around the layers (verification, token plan, head
norm with rotation, prompt attention), made on the host before anything is enqueued."""
import ctypes as C

import pytest
import torch

import csa2_sparse_attention_decode_b200 as csa2

G = C.c_void_p(256 * 100)                      # never dereferenced: the calls below are refused


def test_verify_refusals():
    f = csa2.lib.csa2_verify

    def call(batch=2, k=2, vocab=100, target=G, probs=G, draft=G, n_draft=G, u=G, acc=G, tok=G, err=G):
        return f(batch, k, vocab, target, probs, draft, n_draft, u, acc, tok, err, None)

    for kw in ({"batch": 0}, {"batch": 65536}, {"k": -1}, {"k": csa2.MAX_DRAFT + 1}, {"vocab": 0},
               {"vocab": (1 << 28) + 1}, {"target": None}, {"draft": None}, {"n_draft": None}, {"u": None},
               {"acc": None}, {"tok": None}, {"err": None}):
        assert call(**kw) == 1, kw


def test_plan_refusals():
    f = csa2.lib.csa2_plan_tokens
    H = C.c_void_p(256 * 200)
    ptrs = ["n_tokens", "n_new", "m", "table", "free", "n_free", "n_free_out", "cu", "req", "pos", "slot", "err"]

    def call(batch=2, max_pages=4, n_pages=16, max_new=8, **kw):
        p = {n: kw.get(n, H if n == "n_free_out" else G) for n in ptrs}
        return f(batch, max_pages, n_pages, max_new, *[p[n] for n in ptrs], None)

    for kw in ({"batch": 0}, {"batch": csa2.PLAN_MAX_BATCH + 1}, {"max_pages": 0}, {"max_pages": (1 << 24) + 1},
               {"n_pages": 0}, {"n_pages": 1 << 25}, {"max_new": -1}, {"n_free_out": G}):
        assert call(**kw) == 1, kw
    for n in ptrs:
        assert call(**{n: None}) == 1, n


def test_norm_rope_refusals():
    f = csa2.lib.csa2_norm_rope
    odd = C.c_void_p(256 * 100 + 8)

    def call(n=4, dim=512, heads=64, q=G, qs=64 * 512, qw=G, qo=G, kv=1, k=G, ks=512, kw=G, ko=G, kf=G, pos=G,
             freq=G, rot=64, eps=1e-6, flags=0):
        return f(n, dim, heads, q, qs, qw, qo, kv, k, ks, kw, ko, kf, pos, freq, rot, eps, flags, None, None)

    for bad in ({"n": -1}, {"dim": 96}, {"heads": -1}, {"heads": 1025}, {"kv": -1}, {"kv": 1025},
                {"heads": 0, "kv": 0}, {"rot": 8}, {"rot": 48}, {"rot": 1024}, {"eps": -1.0}, {"eps": float("nan")},
                {"flags": 8}, {"q": None}, {"qw": None}, {"qo": None}, {"qs": 64 * 512 - 8}, {"qs": 64 * 512 + 4},
                {"k": None}, {"kw": None}, {"ko": None, "kf": None}, {"ks": 504}, {"ks": 516}, {"pos": None},
                {"freq": None}, {"q": odd}, {"qo": odd}, {"k": odd}, {"ko": odd}, {"kf": odd}, {"qw": odd}):
        assert call(**bad) == 1, bad
    # in place over rows that lie apart
    assert call(q=G, qo=G, qs=65 * 512) == 1
    assert call(qo=C.c_void_p(256 * 300), k=G, ko=G, ks=1024) == 1
    assert call(n=0) == 0                      # nothing to do, nothing enqueued


def test_prompt_attend_refusals():
    f = csa2.lib.csa2_prompt_attend
    odd = C.c_void_p(256 * 100 + 8)

    def call(batch=2, cu_q=G, cu_k=G, n_q=100, n_k=300, heads=64, q=G, lat=G, stride=512, window=0, scale=0.1, out=G,
             f32=0, lse=None, err=G, ws=G, ws_bytes=1 << 30):
        return f(batch, cu_q, cu_k, n_q, n_k, heads, q, lat, stride, window, scale, out, f32, lse, err, ws, ws_bytes,
                 None)

    need = csa2.csa2_prompt_workspace_bytes(100, 64, 300)
    for bad in ({"batch": 0}, {"n_q": -1}, {"n_k": -1}, {"heads": 0}, {"heads": 129}, {"window": -1}, {"cu_q": None},
                {"cu_k": None}, {"q": None}, {"lat": None}, {"out": None}, {"err": None}, {"ws": None}, {"q": odd},
                {"lat": odd}, {"out": odd}, {"ws": odd}, {"stride": 511}, {"stride": 516}, {"stride": 504},
                {"ws_bytes": need - 1}, {"n_q": 1 << 25}, {"n_k": (1 << 31) - 1}):
        assert call(**bad) == 1, bad
    assert call(n_q=0, q=None, out=None, ws=None) == 0
    assert csa2.csa2_prompt_workspace_bytes(0, 64, 300) == 0 == csa2.csa2_prompt_workspace_bytes(10, 129, 300)
    assert csa2.csa2_prompt_workspace_bytes(1, 64, 128) == 256 == csa2.csa2_prompt_workspace_bytes(100000, 64, 100000)


def test_bindings_refuse_wrong_types_shapes_and_places():
    f32, i32 = torch.float32, torch.int32
    t = torch.zeros(2, 3, 10)
    with pytest.raises(ValueError, match="device tensors"):
        csa2.csa2_verify(t, None, torch.zeros(2, 2, dtype=i32), torch.zeros(2, dtype=i32), torch.zeros(2, 3),
                         torch.zeros(2, dtype=i32), torch.zeros(2, 3, dtype=i32), torch.zeros(1, dtype=i32))
    with pytest.raises(ValueError, match="target"):
        csa2.csa2_verify(t.double(), None, None, None, None, None, None, None)
    with pytest.raises(ValueError, match="n_tokens"):
        csa2.csa2_plan_tokens(torch.zeros(3, dtype=i32), None, None, torch.zeros(2, 4, dtype=i32),
                              torch.zeros(9, dtype=i32), None, None, None, torch.zeros(5, dtype=i32), None, None, None)
    with pytest.raises(ValueError, match="q or k"):
        csa2.csa2_norm_rope(None, None, None, None, None, None, 1e-6, None, None)
    q = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="bfloat16"):
        csa2.csa2_norm_rope(q.to(f32), None, None, None, None, None, 1e-6, None, None)
    with pytest.raises(ValueError, match="contiguous"):
        csa2.csa2_norm_rope(q.transpose(1, 2), None, None, None, None, None, 1e-6, None, None)
    with pytest.raises(ValueError, match="device tensors"):
        csa2.csa2_norm_rope(q, None, None, None, None, None, 1e-6, None, None)

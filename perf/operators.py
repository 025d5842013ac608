"""What a serving program runs around the CSA2 layers of a step, as measured
cases: drafted tokens verified, pages and slots planned for the tokens that
stay, queries and latents normalised and rotated, and the prompt's attention
over the shared latent.

Each case runs one operator once.  With ``own`` false it runs in plain torch;
with ``own`` true through this repository's calls of include/csa2.h.

Cases (what each stands for):
  plan-*    pages and slots of a batch: one decode step of 64 ragged requests,
            the prompts of 64 requests arriving together, a step after
            verification in which some requests drop tokens and some finish.
  norm-*    64 query heads and the latent of 512 channels: the tokens of one
            decode step, and of a prompt; the 32 indexer heads of 128 channels
            with the indexer key, channels paired in halves.
  attend-*  one token of one request over a long past; a decode batch with
            ragged pasts; packed prompts in a layer that sees a 128-token
            window; one prompt in a layer that sees everything before it.
  verify-*  two drafted tokens for 64 requests; five for 8 requests from a
            drafter that proposes without probabilities.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
LATENT = 512
PAGE = 64
VERIFY_FACTOR = 0.7


# ---------------------------------------------------------------- cases
# Lengths of a packed batch are written as one text: "5000 1 129".
def _text(lengths):
    return " ".join(str(n) for n in lengths)


def _ints(text):
    return [int(n) for n in text.split()]


def listed():
    return [
        {"name": "plan-decode-64", "op": "plan", "batch": 64, "past_lo": 4096, "past_hi": 1 << 20,
         "new_lo": 1, "new_hi": 1, "drop": 0.0},
        {"name": "plan-prompt-64", "op": "plan", "batch": 64, "past_lo": 0, "past_hi": 0,
         "new_lo": 500, "new_hi": 16384, "drop": 0.0},
        {"name": "plan-verified-300", "op": "plan", "batch": 300, "past_lo": 1, "past_hi": 32768,
         "new_lo": 1, "new_hi": 6, "drop": 0.25},
        {"name": "norm-decode-64", "op": "norm", "n": 64, "heads": 64, "kv": 1, "dim": 512, "rot": 64,
         "halves": False, "f32": True, "pad": 0},
        {"name": "norm-prompt-8192", "op": "norm", "n": 8192, "heads": 64, "kv": 1, "dim": 512, "rot": 64,
         "halves": False, "f32": False, "pad": 0},
        {"name": "norm-indexer-16381", "op": "norm", "n": 16381, "heads": 32, "kv": 1, "dim": 128, "rot": 128,
         "halves": True, "f32": True, "pad": 128},
        {"name": "attend-token-131072", "op": "attend", "heads": 64, "new": "1", "past": "131071", "window": 0,
         "f32": False},
        {"name": "attend-decode-32", "op": "attend", "heads": 64, "new": _text([1] * 32),
         "past": _text(257 * (i + 1) * (i % 4 + 1) for i in range(32)), "window": 0, "f32": False},
        {"name": "attend-window-16k", "op": "attend", "heads": 64,
         "new": "5000 1 129 4096 777 2000 64 4317", "past": "0 100 0 0 128 0 3 0", "window": 128,
         "f32": False},
        {"name": "attend-causal-6000", "op": "attend", "heads": 64, "new": "6000", "past": "0", "window": 0,
         "f32": False},
        {"name": "verify-64x2", "op": "verify", "batch": 64, "draft": 2, "vocab": 131072, "probs": True},
        {"name": "verify-8x5", "op": "verify", "batch": 8, "draft": 5, "vocab": 100003, "probs": False},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["plan", "norm", "attend", "verify"])
    if op == "plan":
        new_hi = rng.choice([1, 6, _log(rng, 7, 8192)])
        return {"op": op, "batch": _log(rng, 1, 512) if new_hi < 7 else _log(rng, 1, 64), "past_lo": 0,
                "past_hi": _log(rng, 16, 1 << 18), "new_lo": rng.choice([0, 1]), "new_hi": new_hi,
                "drop": rng.choice([0.0, 0.3])}
    if op == "norm":
        dim = rng.choice([64, 128, 256, 512])
        heads = rng.choice([0, 1, 3, 16, 32, 40, 64, 128])
        kv = rng.choice([1, 1, 2, 5]) if heads else 1
        rows = 8192 * 65 * 512 // ((heads + kv) * dim)
        rot = rng.choice([r for r in (0, 16, 32, 64, 128, 256, 512) if r <= dim])
        return {"op": op, "n": _log(rng, 1, min(rows, 20000)), "heads": heads, "kv": kv, "dim": dim, "rot": rot,
                "halves": rng.random() < 0.5, "f32": rng.random() < 0.5, "pad": rng.choice([0, 8, 512])}
    if op == "verify":
        k = rng.choice([0, 1, 2, 3, 7])
        return {"op": op, "batch": _log(rng, 1, 64), "draft": k, "vocab": _log(rng, 100, 131072),
                "probs": rng.random() < 0.6}
    heads = rng.choice([1, 8, 16, 33, 40, 64, 100, 128])
    kind = rng.choice(["token", "window", "prompt"])
    batch = _log(rng, 1, 16)
    if kind == "token":
        new = [rng.choice([0, 1, 1, 1, 2]) for _ in range(batch)]
        if sum(new) == 0:
            new[0] = 1
        past = [_log(rng, 1, 131072 // batch) for _ in range(batch)]
        window = rng.choice([0, 0, 128, 1000])
    elif kind == "window":
        new = [_log(rng, 1, 8192 // batch) for _ in range(batch)]
        past = [rng.choice([0, rng.randrange(200)]) for _ in range(batch)]
        window = rng.choice([1, 64, 128, 128, 500])
    else:
        new = [_log(rng, 1, 2500 // batch + 1) for _ in range(batch)]
        past = [rng.choice([0, 0, _log(rng, 1, 2000)]) for _ in range(batch)]
        window = 0
    return {"op": op, "heads": heads, "new": _text(new), "past": _text(past), "window": window, "f32": rng.random() < 0.25}


# ---------------------------------------------------------------- inputs
def _i32(x):
    return torch.as_tensor(np.asarray(x, np.int32), device=DEV)


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _plan_lengths(case, seed):
    r = np.random.default_rng(seed)
    B = case["batch"]

    def span(lo, hi):
        if hi <= lo:
            return np.full(B, lo, np.int64)
        return np.clip(np.exp(r.uniform(np.log(lo + 1), np.log(hi + 1), B)).astype(np.int64) - 1, lo, hi)

    past, new = span(case["past_lo"], case["past_hi"]), span(case["new_lo"], case["new_hi"])
    m = 1 + (r.random(B) < 0.25).astype(np.int64)
    gone = r.random(B) < case["drop"]
    back = np.where(r.random(B) < 0.3, past, np.minimum(past, r.integers(0, 200, B)))
    return r, past, np.where(gone, -back, new), m


def _prepare_plan(case, seed):
    r, past, new, m = _plan_lengths(case, seed)
    B = case["batch"]
    owned = -(-(past // m) // PAGE)
    max_pages = -(-(case["past_hi"] + case["new_hi"]) // PAGE) + 1       # the longest a request may get
    n_pages = B * max_pages
    perm = r.permutation(n_pages)
    table = np.full((B, max_pages), -1, np.int32)
    at = 0
    for b in range(B):
        table[b, :owned[b]] = perm[at:at + owned[b]]
        at += owned[b]
    free = np.full(n_pages, -1, np.int32)
    free[:n_pages - at] = perm[at:]
    room = B * case["new_hi"] + 5
    return {"n_tokens": _i32(past), "n_new": _i32(new), "m": _i32(m), "page_table": _i32(table),
            "free_pages": _i32(free), "n_free": _i32([n_pages - at]), "n_free_out": _i32([0]),
            "cu_new": _i32(np.zeros(B + 1)), "token_req": _i32(np.full(room, -7)),
            "token_pos": _i32(np.full(room, -7)), "token_slot": _i32(np.full(room, -7)), "error": _i32([0])}


def _prepare_norm(case, seed):
    g = _gen(seed)
    n, H, G, D, R = case["n"], case["heads"], case["kv"], case["dim"], case["rot"]
    # one projection's output holds every head of a token side by side
    wide = (H + G) * D + case["pad"]
    x = (torch.randn(n, wide, generator=g, device=DEV) *
         torch.exp(0.5 * torch.randn(wide, generator=g, device=DEV))).to(torch.bfloat16)
    st = {"x": x, "q": x[:, :H * D].view(n, H, D) if H else None, "k": x[:, H * D:(H + G) * D].view(n, G, D),
          "pos": torch.randint(0, 1 << 20, (n,), generator=g, device=DEV, dtype=torch.int32),
          "inv_freq": None, "q_weight": None, "k_weight": 1 + 0.1 * torch.randn(D, generator=g, device=DEV),
          "q_out": None, "k_out": torch.empty(n, G, D, dtype=torch.bfloat16, device=DEV), "k_f32": None}
    if H:
        st["q_weight"] = 1 + 0.1 * torch.randn(D, generator=g, device=DEV)
        st["q_out"] = torch.empty(n, H, D, dtype=torch.bfloat16, device=DEV)
    if R:
        st["inv_freq"] = (10000.0 ** (-torch.arange(0, R, 2, dtype=torch.float64) / R)).float().to(DEV)
    if case["f32"]:
        st["k_f32"] = torch.empty(n, G, D, dtype=torch.float32, device=DEV)
    return st


def _prepare_attend(case, seed):
    g = _gen(seed)
    H = case["heads"]
    new = _ints(case["new"])
    kv = [a + b for a, b in zip(new, _ints(case["past"]))]
    nq, nk = sum(new), sum(kv)
    chan = torch.exp(0.5 * torch.randn(LATENT, generator=g, device=DEV))
    st = {"q": torch.randn(nq, H, LATENT, generator=g, device=DEV, dtype=torch.bfloat16),
          "lat": (torch.randn(nk, LATENT, generator=g, device=DEV) * chan).to(torch.bfloat16),
          "cu_q": _i32(np.concatenate([[0], np.cumsum(new)])), "cu_k": _i32(np.concatenate([[0], np.cumsum(kv)])),
          "out": torch.empty(nq, H, LATENT, dtype=torch.float32 if case["f32"] else torch.bfloat16, device=DEV),
          "lse": torch.empty(nq, H, dtype=torch.float32, device=DEV), "error": _i32([0]), "ws": None}
    if own:
        import csa2_sparse_attention_decode_b200 as csa2
        st["ws"] = torch.empty(csa2.csa2_prompt_workspace_bytes(nq, H, nk), dtype=torch.uint8, device=DEV)
    return st


def _prepare_verify(case, seed):
    g = _gen(seed)
    B, K, V = case["batch"], case["draft"], case["vocab"]
    base = 3.0 * torch.randn(B, K + 1, V, generator=g, device=DEV)
    target = torch.softmax(base, -1)
    probs = None
    if case["probs"]:
        probs = torch.softmax(base[:, :K] + VERIFY_FACTOR * torch.randn(B, K, V, generator=g, device=DEV), -1)
    # what the drafter drew from its own distribution (a point mass: its best guess)
    gum = -torch.log(-torch.log(torch.rand(B, K, V, generator=g, device=DEV).clamp(1e-12, 1 - 1e-7)))
    draft = (torch.log(probs if probs is not None else target[:, :K]) + gum).argmax(-1).to(torch.int32) if K else \
        torch.zeros(B, 0, dtype=torch.int32, device=DEV)
    del base, gum
    nd = torch.randint(0, K + 1, (B,), generator=g, device=DEV, dtype=torch.int32)
    n_draft = torch.where(torch.rand(B, generator=g, device=DEV) < 0.8, torch.full_like(nd, K), nd)
    return {"target": target, "probs": probs, "draft": draft, "n_draft": n_draft,
            "u": torch.rand(B, K + 1, generator=g, device=DEV), "n_accepted": _i32(np.zeros(B)),
            "tokens": _i32(np.zeros((B, K + 1))), "error": _i32([0])}


def prepare(case, seed):
    st = {"plan": _prepare_plan, "norm": _prepare_norm, "attend": _prepare_attend,
          "verify": _prepare_verify}[case["op"]](case, seed)
    st["case"] = case
    return st


# ---------------------------------------------------------------- plain forms
def _plain_plan(s):
    past, new, m = s["n_tokens"].long(), s["n_new"].long(), s["m"].long()
    table, free, n_free = s["page_table"], s["free_pages"], s["n_free"].long()
    B, width = table.shape
    owned = (past // m + PAGE - 1) // PAGE
    need = ((past + new) // m + PAGE - 1) // PAGE
    col = torch.arange(width, device=DEV)[None, :]
    # released pages go on the stack in request order, then pages are taken off its top
    rel = (owned - need).clamp_min(0)
    rel_at = torch.cumsum(rel, 0) - rel
    stack = torch.cat([free, torch.zeros(1, dtype=torch.int32, device=DEV)])
    is_rel = (col >= need[:, None]) & (col < owned[:, None])
    dst = torch.where(is_rel, n_free + rel_at[:, None] + col - need[:, None], free.numel())
    stack = stack.scatter(0, dst.flatten(), table.flatten())[:-1]
    top = n_free + rel.sum()
    get = (need - owned).clamp_min(0)
    get_at = torch.cumsum(get, 0) - get
    ok = (get == 0) | (get_at + get <= top)
    get, new = get * ok, (new * ok).clamp_min(0)
    is_get = (col >= owned[:, None]) & (col < (owned + get)[:, None])
    src = (top - 1 - (get_at[:, None] + col - owned[:, None])).clamp(0, free.numel() - 1)
    table = torch.where(is_get, stack[src], table)
    cu = torch.cat([torch.zeros(1, dtype=torch.long, device=DEV), torch.cumsum(new, 0)])
    i = torch.arange(s["token_req"].numel(), device=DEV)
    live = i < cu[-1]
    req = torch.searchsorted(cu[1:].contiguous(), i, right=True).clamp_max(B - 1)
    pos = past[req] + i - cu[req]
    e = pos // m[req]
    slot = table[req, (e // PAGE).clamp_max(width - 1)].long() * PAGE + e % PAGE
    slot = torch.where((m[req] == 2) & (pos % 2 == 0), -1, slot)
    return (table, stack, (top - get.sum()).int(), cu.int(), torch.where(live, req, s["token_req"]).int(),
            torch.where(live, pos, s["token_pos"]).int(), torch.where(live, slot, s["token_slot"]).int())


def _plain_rows(x, w, pos, inv_freq, halves, eps):
    y = x.float()
    y = y * torch.rsqrt((y * y).mean(-1, keepdim=True) + eps) * w
    if inv_freq is None:
        return y
    R = 2 * inv_freq.numel()
    ang = (pos.double()[:, None] * inv_freq.double()[None, :])[:, None, :]
    c, sn = torch.cos(ang).float(), torch.sin(ang).float()
    tail = y[..., -R:]
    a, b = (tail[..., :R // 2], tail[..., R // 2:]) if halves else (tail[..., 0::2], tail[..., 1::2])
    ra, rb = a * c - b * sn, a * sn + b * c
    tail = torch.cat([ra, rb], -1) if halves else torch.stack([ra, rb], -1).flatten(-2)
    return torch.cat([y[..., :-R], tail], -1)


def _plain_norm(s):
    h = s["case"]["halves"]
    out = []
    if s["q"] is not None:
        out.append(_plain_rows(s["q"], s["q_weight"], s["pos"], s["inv_freq"], h, 1e-6).to(torch.bfloat16))
    k = _plain_rows(s["k"], s["k_weight"], s["pos"], s["inv_freq"], h, 1e-6)
    out.append(k.to(torch.bfloat16))
    if s["k_f32"] is not None:
        out.append(k)
    return tuple(out)


def _plain_attend(s, chunk=256):
    case, q, lat = s["case"], s["q"], s["lat"]
    H, W = case["heads"], case["window"]
    scale = 1.0 / math.sqrt(LATENT)
    out, lse = torch.zeros(q.shape, device=DEV), torch.full(q.shape[:2], -math.inf, device=DEV)
    q0 = k0 = 0
    for n, p in zip(_ints(case["new"]), _ints(case["past"])):
        for a in range(0, n, chunk):
            b = min(n, a + chunk)
            lo = max(0, p + a + 1 - W) if W else 0
            kv = lat[k0 + lo:k0 + p + b].float()
            sc = torch.matmul(q[q0 + a:q0 + b].float(), kv.t()) * scale                # [rows, H, keys]
            i = torch.arange(a, b, device=DEV)[:, None] + p
            j = torch.arange(lo, p + b, device=DEV)[None, :]
            see = (j <= i) & (j > i - W) if W else j <= i
            sc = sc.masked_fill(~see[:, None, :], -math.inf)
            mx = sc.amax(-1, keepdim=True)
            e = torch.exp(sc - mx)
            den = e.sum(-1, keepdim=True)
            out[q0 + a:q0 + b] = torch.matmul(e, kv) / den
            lse[q0 + a:q0 + b] = (mx + torch.log(den))[..., 0]
        q0, k0 = q0 + n, k0 + n + p
    return out.to(s["out"].dtype), lse


def _plain_verify(s):
    t, d, u = s["target"], s["draft"].long(), s["u"].double()
    B, K1, V = t.shape
    K = K1 - 1
    i = torch.arange(K, device=DEV)[None, :]
    p = t[:, :K].gather(2, d[..., None])[..., 0].double()
    q = torch.ones_like(p) if s["probs"] is None else s["probs"].gather(2, d[..., None])[..., 0].double()
    take = (u[:, :K] * q < p) & (i < s["n_draft"][:, None])
    n = torch.cumprod(take.long(), 1).sum(1)
    rows = torch.arange(B, device=DEV)
    w = t[rows, n].double()
    if K:
        rejected = n < s["n_draft"]
        at = n.clamp_max(K - 1)
        if s["probs"] is None:
            q_row = torch.zeros_like(w).scatter(1, d[rows, at][:, None], 1.0)
        else:
            q_row = s["probs"][rows, at].double()
        r = torch.where(rejected[:, None], (w - q_row).clamp_min(0), w)
        w = torch.where(r.sum(1, keepdim=True) > 0, r, w)
    cdf = torch.cumsum(w, 1)
    x = torch.searchsorted(cdf, u[:, K:] * cdf[:, -1:], right=True)[:, 0].clamp_max(V - 1)
    col = torch.arange(K1, device=DEV)[None, :]
    full = torch.cat([d, torch.zeros(B, 1, dtype=torch.long, device=DEV)], 1)
    tok = torch.where(col < n[:, None], full, torch.where(col == n[:, None], x[:, None], -1))
    return n.int(), tok.int()


# ---------------------------------------------------------------- one pass
def run(s):
    op = s["case"]["op"]
    if not own:
        return {"plan": _plain_plan, "norm": _plain_norm, "attend": _plain_attend, "verify": _plain_verify}[op](s)
    import csa2_sparse_attention_decode_b200 as csa2
    if op == "plan":
        csa2.csa2_plan_tokens(s["n_tokens"], s["n_new"], s["m"], s["page_table"], s["free_pages"], s["n_free"],
                              s["n_free_out"], s["cu_new"], s["token_req"], s["token_pos"], s["token_slot"],
                              s["error"])
        return (s["page_table"], s["free_pages"], s["n_free_out"], s["cu_new"], s["token_req"], s["token_pos"],
                s["token_slot"])
    if op == "norm":
        flags = csa2.ROPE_HALVES if s["case"]["halves"] else 0
        csa2.csa2_norm_rope(s["q"], s["k"], s["pos"], s["inv_freq"], s["q_weight"], s["k_weight"], 1e-6, s["q_out"],
                            s["k_out"], s["k_f32"], flags=flags)
        return tuple(x for x in (s["q_out"], s["k_out"], s["k_f32"]) if x is not None)
    if op == "attend":
        csa2.csa2_prompt_attend(s["q"], s["lat"], s["cu_q"], s["cu_k"], s["case"]["window"],
                                1.0 / math.sqrt(LATENT), s["out"], s["lse"], s["error"], s["ws"])
        return s["out"], s["lse"]
    csa2.csa2_verify(s["target"], s["probs"], s["draft"], s["n_draft"], s["u"], s["n_accepted"], s["tokens"],
                     s["error"])
    return s["n_accepted"], s["tokens"]


# ---------------------------------------------------------------- the definition in 64 bits
def _exact_plan(case, s):
    past, new, m = (s[k].cpu().numpy().astype(int) for k in ("n_tokens", "n_new", "m"))
    table, stack = s["page_table"].cpu().numpy().copy(), s["free_pages"].cpu().numpy().copy()
    top = int(s["n_free"][0])

    def pages(tok, ratio):
        return -(-(tok // ratio) // PAGE)

    for b in range(len(past)):
        for j in range(pages(past[b] + new[b], m[b]), pages(past[b], m[b])):
            stack[top] = table[b, j]
            top += 1
    cu, left = [0], top
    for b in range(len(past)):
        a, z = pages(past[b], m[b]), pages(past[b] + new[b], m[b])
        if z > a:
            for j in range(a, z):
                left -= 1
                table[b, j] = stack[left]
        cu.append(cu[-1] + max(0, int(new[b])))
    req, pos, slot = (s[k].cpu().numpy().copy() for k in ("token_req", "token_pos", "token_slot"))
    for b in range(len(past)):
        t = np.arange(past[b], past[b] + cu[b + 1] - cu[b])
        at = slice(cu[b], cu[b + 1])
        req[at], pos[at] = b, t
        e = t // m[b]
        slot[at] = np.where((m[b] == 2) & (t % 2 == 0), -1, table[b, e // PAGE] * PAGE + e % PAGE)
    return table, stack, np.array([left], np.int32), np.array(cu, np.int32), req, pos, slot


def _exact_norm(case, s):
    def rows(x, w):
        y = x.double()
        y = y / torch.sqrt(y.pow(2).sum(-1, keepdim=True) / y.shape[-1] + float(np.float32(1e-6))) * w.double()
        if s["inv_freq"] is None:
            return y
        R = 2 * s["inv_freq"].numel()
        z = torch.polar(torch.ones(1, dtype=torch.float64, device=DEV),
                        s["pos"].double()[:, None] * s["inv_freq"].double())[:, None, :]
        t = y[..., y.shape[-1] - R:]
        t = t.reshape(*t.shape[:-1], 2, R // 2).transpose(-1, -2) if case["halves"] else \
            t.reshape(*t.shape[:-1], R // 2, 2)
        t = torch.view_as_real(torch.view_as_complex(t.contiguous()) * z)
        y[..., y.shape[-1] - R:] = (t.transpose(-1, -2) if case["halves"] else t).reshape(*y.shape[:-1], R)
        return y

    out = [rows(s["q"], s["q_weight"])] if s["q"] is not None else []
    k = rows(s["k"], s["k_weight"])
    return tuple(out + [k] + ([k] if s["k_f32"] is not None else []))


def _exact_attend(case, s):
    q, lat, H, W = s["q"], s["lat"], case["heads"], case["window"]
    out = torch.zeros(q.shape, dtype=torch.float64, device=DEV)
    lse = torch.zeros(q.shape[:2], dtype=torch.float64, device=DEV)
    cq, ck = s["cu_q"].tolist(), s["cu_k"].tolist()
    for b in range(len(cq) - 1):
        past = (ck[b + 1] - ck[b]) - (cq[b + 1] - cq[b])
        for t in range(cq[b], cq[b + 1], 64):
            e = min(t + 64, cq[b + 1])
            last = ck[b] + past + torch.arange(t - cq[b], e - cq[b], device=DEV)     # each token's own key
            first = torch.clamp(last - W + 1, min=ck[b]) if W else torch.full_like(last, ck[b])
            base, end = int(first[0]), int(last[-1]) + 1
            keys = lat[base:end].double()
            sc = (q[t:e].reshape(-1, LATENT).double() @ keys.T).view(e - t, H, -1) / math.sqrt(LATENT)
            at = torch.arange(base, end, device=DEV)
            sc[((at < first[:, None]) | (at > last[:, None]))[:, None, :].expand_as(sc)] = -math.inf
            lse[t:e] = torch.logsumexp(sc, -1)
            out[t:e] = torch.exp(sc - lse[t:e, :, None]) @ keys
    return out, lse


def _exact_verify(case, s):
    t, d, nd, u = (s[k].cpu().numpy() for k in ("target", "draft", "n_draft", "u"))
    pr = None if s["probs"] is None else s["probs"].cpu().numpy()
    B, K = d.shape
    tok, acc = np.full((B, K + 1), -1, np.int32), np.zeros(B, np.int32)
    for b in range(B):
        n = 0
        while n < nd[b]:
            qx = 1.0 if pr is None else float(pr[b, n, d[b, n]])
            if not float(u[b, n]) * qx < float(t[b, n, d[b, n]]):
                break
            tok[b, n] = d[b, n]
            n += 1
        w = t[b, n].astype(np.float64)
        if n < nd[b]:
            if pr is None:
                r = w.copy()
                r[d[b, n]] = max(0.0, r[d[b, n]] - 1.0)
            else:
                r = np.maximum(w - pr[b, n], 0.0)
            w = r if r.sum() > 0 else w
        c = np.cumsum(w)
        tok[b, n] = int(np.argmax(c > float(u[b, K]) * c[-1]))
        acc[b] = n
    return acc, tok


def exact(case, seed):
    if case["op"] == "attend" and work(case)["flops"] > 6e12:
        return None
    s = prepare(case, seed)
    return {"plan": _exact_plan, "norm": _exact_norm, "attend": _exact_attend, "verify": _exact_verify}[case["op"]](
        case, s)


# ---------------------------------------------------------------- work
def work(case):
    op = case["op"]
    if op == "plan":
        # lengths in; table entries of new pages, and request, position and slot of each new token, out
        B = case["batch"]
        lo, hi = case["new_lo"], case["new_hi"]
        mean = lo if hi <= lo else (hi - lo) / math.log((hi + 1) / (lo + 1))
        tok = B * (1 - case["drop"]) * mean
        return {"bytes": int(16 * B + 12 * tok + 8 * tok / PAGE), "flops": int(10 * tok)}
    if op == "norm":
        x = case["n"] * (case["heads"] + case["kv"]) * case["dim"]
        kf = case["n"] * case["kv"] * case["dim"] * 4 if case["f32"] else 0
        return {"bytes": 4 * x + kf + 4 * case["n"], "flops": 8 * x}
    if op == "verify":
        # the row sampled from, and the drafter's row where a token was refused
        rows = 2 if case["probs"] and case["draft"] else 1
        return {"bytes": case["batch"] * case["vocab"] * 4 * rows, "flops": case["batch"] * case["vocab"] * 3}
    H, W = case["heads"], case["window"]
    nq = sum(_ints(case["new"]))
    nk = nq + sum(_ints(case["past"]))
    pairs = 0
    for n, p in zip(_ints(case["new"]), _ints(case["past"])):
        full = n * p + n * (n + 1) // 2                      # keys 0 .. p + i of token i
        if W:
            c = max(0, n + p - W)                            # tokens whose window leaves keys out
            c0 = max(0, p - W)
            full -= c * (c + 1) // 2 - c0 * (c0 + 1) // 2
        pairs += full
    io = nq * H * LATENT * (2 + (4 if case["f32"] else 2)) + nk * LATENT * 2 + nq * H * 4
    return {"bytes": io, "flops": pairs * H * LATENT * 4}

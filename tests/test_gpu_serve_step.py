"""The calls around the layers used together, as a serving program does: a
prompt's pages, norm, attention and cache entries, then decode steps with
drafted tokens, eagerly and replayed from one captured graph."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

H, IDX, V, SCALE = 16, 32, 5000, 1.0 / math.sqrt(512.0)
M = [1, 2, 1]
PROMPTS = [700, 389, 64]
N_PAGES = 64


def _csa2():
    import csa2_sparse_attention_decode_b200 as csa2
    return csa2


def _i32(x):
    return torch.as_tensor(x, dtype=torch.int32, device="cuda")


class Server:
    """Three requests over one pool; `pages`: how the free pages lie on the stack."""

    def __init__(self, pages):
        csa2 = _csa2()
        B = len(M)
        self.table = torch.full((B, 16), -1, dtype=torch.int32, device="cuda")
        self.cache = csa2.Cache(self.table, N_PAGES, M)
        assert self.cache.page_table.data_ptr() == self.table.data_ptr()       # the plan's pages are the cache's
        self.free, self.n_free, self.n_free_out = _i32(pages), _i32([N_PAGES]), _i32([0])
        self.cu, self.n_new = _i32([0] * (B + 1)), _i32([0] * B)
        g = torch.Generator(device="cuda").manual_seed(3)
        self.wq, self.wk = (1 + 0.1 * torch.randn(512, generator=g, device="cuda") for _ in range(2))
        self.freq = (10000.0 ** (-torch.arange(0, 64, 2, dtype=torch.float64) / 64)).float().cuda()
        self.ws = csa2.workspace(self.cache)
        self.topk = torch.empty(B, 512, dtype=torch.int32, device="cuda")

    def plan(self, rows):
        csa2 = _csa2()
        csa2.csa2_plan_tokens(self.cache.n_tokens, self.n_new, self.cache.m, self.table, self.free, self.n_free,
                              self.n_free_out, self.cu, *rows, self.cache.error)
        self.n_free.copy_(self.n_free_out)

    def prompt(self, x, key, gate):
        """x [n, H + 1, 512]: queries and latent of every prompt token, packed."""
        csa2 = _csa2()
        n = x.shape[0]
        self.n_new.copy_(_i32(PROMPTS))
        rows = [torch.full((n + 9,), -7, dtype=torch.int32, device="cuda") for _ in range(3)]
        self.plan(rows)
        q, lat = torch.empty_like(x[:, :H]), torch.empty_like(x[:, H:])
        lat32 = torch.empty(n, 1, 512, device="cuda")
        csa2.csa2_norm_rope(x[:, :H], x[:, H:], rows[1][:n], self.freq, self.wq, self.wk, 1e-6, q, lat, lat32)
        out = torch.empty_like(q)
        ws = torch.empty(csa2.csa2_prompt_workspace_bytes(n, H, n), dtype=torch.uint8, device="cuda")
        csa2.csa2_prompt_attend(q, lat[:, 0], self.cu, self.cu, csa2.SWA, SCALE, out, None, self.cache.error, ws)
        cu = self.cu.tolist()
        for b in range(len(M)):
            csa2.csa2_prefill(self.cache, b, 0, PROMPTS[b], lat32[cu[b]:cu[b + 1], 0], key[cu[b]:cu[b + 1]],
                              gate[cu[b]:cu[b + 1]])
        return rows, q, lat, out

    def decode(self, s):
        """One step from the static inputs s: verify the draft, plan, rotate, append, select, attend."""
        csa2 = _csa2()
        csa2.csa2_verify(s["target"], s["probs"], s["draft"], s["n_draft"], s["u"], s["acc"], s["tokens"],
                         self.cache.error)
        torch.add(s["acc"], 1, out=self.n_new)                 # the kept draft and the drawn token
        self.plan(s["rows"])
        # rows of the tokens that came, at their positions: padded to the most there can be
        s["pos"].copy_((self.cache.n_tokens[:, None] + torch.arange(2, device="cuda", dtype=torch.int32)).flatten())
        csa2.csa2_norm_rope(None, s["x"], s["pos"], self.freq, None, self.wk, 1e-6, None, None, s["lat32"])
        csa2.csa2_norm_rope(s["qx"], None, s["pos"][:len(M)], self.freq, self.wq, None, 1e-6, s["q"], None)
        csa2.csa2_append(self.cache, s["lat32"].view(len(M), 2, 512), s["key"], s["gate"], self.n_new)
        csa2.csa2_index(self.cache, csa2.INDEX_FLAT, s["ix"], s["hw"], None, None, self.topk, self.ws)
        csa2.csa2_attend(self.cache, s["q"], self.topk, SCALE, s["out"], self.ws)


def _prompt_inputs():
    g = torch.Generator(device="cuda").manual_seed(1)
    n = sum(PROMPTS)
    return (torch.randn(n, H + 1, 512, generator=g, device="cuda").to(torch.bfloat16),
            torch.randn(n, 128, generator=g, device="cuda"), torch.randn(n, generator=g, device="cuda"))


def _step_inputs(seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    B = len(M)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")             # noqa: E731
    return {"target": torch.softmax(3 * r(B, 2, V), -1), "probs": torch.softmax(3 * r(B, 1, V), -1),
            "draft": torch.randint(0, V, (B, 1), generator=g, device="cuda", dtype=torch.int32),
            "n_draft": _i32([1, 0, 1]), "u": torch.rand(B, 2, generator=g, device="cuda") *
            torch.tensor([1e-3, 1.0], device="cuda"),
            "x": r(2 * B, 1, 512).to(torch.bfloat16), "qx": r(B, H, 512).to(torch.bfloat16),
            "ix": r(B, IDX, 128).to(torch.bfloat16), "hw": torch.rand(B, IDX, generator=g, device="cuda"),
            "key": r(B, 2, 128), "gate": r(B, 2)}


def _outputs():
    B = len(M)
    return {"acc": _i32([0] * B), "tokens": _i32([[0, 0]] * B), "pos": _i32([0] * 2 * B),
            "rows": [torch.full((2 * B,), -7, dtype=torch.int32, device="cuda") for _ in range(3)],
            "lat32": torch.empty(2 * B, 1, 512, device="cuda"),
            "q": torch.empty(B, H, 512, dtype=torch.bfloat16, device="cuda"),
            "out": torch.empty(B, H, 512, device="cuda")}


def _pages(server):
    own = [-(-(int(t) // m) // 64) for t, m in zip(server.cache.n_tokens.tolist(), M)]
    held = [p for b, k in enumerate(own) for p in server.table[b, :k].tolist()]
    return held, server.free[:int(server.n_free)].tolist()


def test_prompts_then_decode_steps():
    csa2 = _csa2()
    x, key, gate = _prompt_inputs()
    shuffled = torch.randperm(N_PAGES, generator=torch.Generator().manual_seed(0)).tolist()
    servers = [Server(shuffled), Server(list(range(N_PAGES)))]
    seen = []
    for s in servers:
        rows, q, lat, out = s.prompt(x, key, gate)
        n = x.shape[0]
        assert (rows[0][n:] == -7).all() and int(s.cu[-1]) == n
        # the prompt's attention over the window, from the definition
        at = 0
        for b, length in enumerate(PROMPTS):
            for t in (0, 1, 63, length - 1):
                k = lat[at + max(0, t - 127):at + t + 1, 0].double()
                w = torch.softmax(q[at + t].double() @ k.T * SCALE, -1)
                ref, mag = w @ k, w @ k.abs()
                # output and weights are rounded to bf16 (2^-8 each); a score is off by up to 512 * 2^-24 of
                # the sum of its products (about 19 * SCALE * 512 / 23 = 16 here), twice: under 2^-10
                assert ((out[at + t].double() - ref).abs() <= 2.0 ** -8 * (ref.abs() + mag) + 2.0 ** -10 * mag).all()
            at += length
        # the slots the plan gave are where the entries lie: codes that are not the pool's zeros
        slots = rows[2][:n]
        done = slots[slots >= 0].long()
        assert done.unique().numel() == done.numel() == sum(t // m for t, m in zip(PROMPTS, M))
        codes = s.cache.pool[:N_PAGES * 16384].view(-1, 256)
        assert codes[done].any(-1).all() and not codes.any(-1).sum() - done.numel()
        results = []
        for step in range(4):
            st = {**_step_inputs(10 + step), **_outputs()}
            s.decode(st)
            results.append((st["acc"].clone(), st["tokens"].clone(), s.topk.clone(), st["out"].clone()))
        held, free = _pages(s)
        assert sorted(held + free) == list(range(N_PAGES))
        assert csa2.csa2_get_device_error(s.cache) == 0
        seen.append(results)
    # where a request's pages lie changes nothing
    for a, b in zip(*seen):
        assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_captured_steps_and_release():
    csa2 = _csa2()
    x, key, gate = _prompt_inputs()
    eager, replayed = Server(list(range(N_PAGES))), Server(list(range(N_PAGES)))
    for s in (eager, replayed):
        s.prompt(x, key, gate)
    static = {**_step_inputs(20), **_outputs()}
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        replayed.decode(static)
    for step in range(12):                     # past a page's border for every request
        fresh = _step_inputs(30 + step)
        for k, v in fresh.items():
            static[k].copy_(v)
        graph.replay()
        st = {**fresh, **_outputs()}
        eager.decode(st)
        for k in ("acc", "tokens", "out"):
            assert torch.equal(static[k], st[k]), (step, k)
        assert torch.equal(replayed.topk, eager.topk) and torch.equal(replayed.table, eager.table)
    # the first request ends: its pages return to the stack and go to nobody twice
    for s in (eager, replayed):
        s.n_new.copy_(torch.stack([-s.cache.n_tokens[0], torch.zeros_like(s.n_new[0]), torch.zeros_like(s.n_new[0])]))
        s.plan(_outputs()["rows"])
        s.cache.n_tokens[0] = 0
        held, free = _pages(s)
        assert sorted(held + free) == list(range(N_PAGES))
        assert csa2.csa2_get_device_error(s.cache) == 0


def test_prompt_attention_on_two_streams_at_once():
    csa2 = _csa2()
    g = torch.Generator(device="cuda").manual_seed(4)
    streams = [torch.cuda.Stream() for _ in range(2)]
    q = torch.randn(40, 64, 512, generator=g, device="cuda").to(torch.bfloat16)
    lat = torch.randn(9000, 512, generator=g, device="cuda").to(torch.bfloat16)
    cu_q, cu_k = _i32([0, 40]), _i32([0, 9000])
    outs = []
    torch.cuda.synchronize()
    for s in [None] + streams:                 # once alone, then both together
        o = (torch.empty_like(q), torch.empty(40, 64, device="cuda"), _i32([0]),
             torch.empty(csa2.csa2_prompt_workspace_bytes(40, 64, 9000), dtype=torch.uint8, device="cuda"))
        outs.append(o)
    torch.cuda.synchronize()
    csa2.csa2_prompt_attend(q, lat, cu_q, cu_k, 0, SCALE, outs[0][0], outs[0][1], outs[0][2], outs[0][3])
    torch.cuda.synchronize()
    for _ in range(5):
        for s, o in zip(streams, outs[1:]):
            csa2.csa2_prompt_attend(q, lat, cu_q, cu_k, 0, SCALE, *o, stream=s)
    torch.cuda.synchronize()
    for o in outs[1:]:
        assert torch.equal(o[0], outs[0][0]) and torch.equal(o[1], outs[0][1]) and int(o[2]) == 0

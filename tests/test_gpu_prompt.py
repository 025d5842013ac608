"""csa2_prompt_attend against the definition in 64 bits: packed prompts,
windows, continued prompts, single tokens over a long past, rows without
keys, latents that are not finite, and tokens behind the last request."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

SCALE = 1.0 / math.sqrt(512.0)
U24, U8 = 2.0 ** -24, 2.0 ** -8                # half steps of f32 and bf16, relative


def _csa2():
    import csa2_sparse_attention_decode_b200 as csa2
    return csa2


def _cu(lengths):
    return torch.tensor([sum(lengths[:i]) for i in range(len(lengths) + 1)], dtype=torch.int32, device="cuda")


def _inputs(seed, new, kv, heads, extra_q=0, extra_k=0, stride=512):
    g = torch.Generator(device="cuda").manual_seed(seed)
    chan = torch.exp(0.5 * torch.randn(512, generator=g, device="cuda"))
    q = torch.randn(sum(new) + extra_q, heads, 512, generator=g, device="cuda").to(torch.bfloat16)
    wide = torch.randn(sum(kv) + extra_k, stride, generator=g, device="cuda")
    wide[:, :512] *= chan
    return q, wide.to(torch.bfloat16)[:, :512]


def _call(q, lat, cu_q, cu_k, window=0, f32=False, scale=SCALE, out=None, lse=None, ws=None, err=None):
    csa2 = _csa2()
    out = torch.full(q.shape, 7.0, dtype=torch.float32 if f32 else torch.bfloat16, device="cuda") if out is None else out
    lse = torch.full(q.shape[:2], 7.0, device="cuda") if lse is None else lse
    err = torch.zeros(1, dtype=torch.int32, device="cuda") if err is None else err
    if ws is None:
        ws = torch.empty(csa2.csa2_prompt_workspace_bytes(q.shape[0], q.shape[1], lat.shape[0]), dtype=torch.uint8,
                         device="cuda")
    csa2.csa2_prompt_attend(q, lat, cu_q, cu_k, window, scale, out, lse, err, ws)
    return out, lse, err


def _ref(q, lat, p, window, scale=SCALE):
    """One request, p latents before its first token: output, lse, sum of weights * |latent| (what rounding a
    weight scales with), and the bound on a score's fp32 error."""
    n = q.shape[0]
    v = lat.double()
    s = torch.einsum("thd,kd->thk", q.double(), v) * scale
    i = torch.arange(n, device="cuda")[:, None] + p
    j = torch.arange(lat.shape[0], device="cuda")[None, :]
    see = (j <= i) & ((j > i - window) if window else torch.ones_like(j <= i))
    s = s.masked_fill(~see[:, None, :], -math.inf)
    lse = torch.logsumexp(s, -1)
    w = torch.exp(s - lse.masked_fill(lse == -math.inf, 0)[..., None])
    err = 512 * U24 * abs(scale) * torch.einsum("thd,kd->thk", q.double().abs(), v.abs())
    err = err.masked_fill(~see[:, None, :], 0).amax(-1)[..., None] if lat.shape[0] else torch.zeros_like(lse)[..., None]
    return torch.einsum("thk,kd->thd", w, v), lse, torch.einsum("thk,kd->thd", w, v.abs()), err


# Output: every weight is off by its rounding (bf16: 2^-8; kept in two parts:
# 2^-16), by the exponential (2^-22) and by its score's error, once in the
# weight and once in their sum; fp32 sums over the keys add 2^-22 more, and
# the output is rounded once.  lse: the score's error, the logarithm (2^-22).
def _check(out, lse, ref, what=""):
    o, l, mag, err = ref
    f32 = out.dtype == torch.float32
    tol = (2.0 ** -16 if f32 else U8) * mag + (2 * err + 2.0 ** -20) * mag + (U24 if f32 else U8) * o.abs() + 1e-30
    bad = ~((out.double() - o).abs() <= tol)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} off, first {bad.nonzero()[0].tolist()}, " \
                          f"worst {float(((out.double() - o).abs() / tol).nan_to_num(1e9).max()):.3g} x"
    none = l == -math.inf
    assert torch.equal(lse == -math.inf, none), what
    assert ((lse.double() - l).abs() <= err[..., 0] + 2.0 ** -20 * (1 + l.abs()))[~none].all(), what


def _check_all(new, past, heads, window=0, f32=False, seed=0, stride=512, extra_q=0, extra_k=0):
    kv = [max(0, n + p) for n, p in zip(new, past)]
    q, lat = _inputs(seed, new, kv, heads, extra_q, extra_k, stride)
    cu_q, cu_k = _cu(new), _cu(kv)
    out, lse, err = _call(q, lat, cu_q, cu_k, window, f32)
    assert int(err) == 0
    a = c = 0
    for b, (n, k, p) in enumerate(zip(new, kv, past)):
        if n:
            _check(out[a:a + n], lse[a:a + n], _ref(q[a:a + n], lat[c:c + k], p, window), f"request {b}")
        a, c = a + n, c + k
    assert (out[a:] == 7).all() and (lse[a:] == 7).all()               # behind the last request: left alone
    return q, lat, cu_q, cu_k, out, lse


@pytest.mark.parametrize("heads", [64, 16, 128, 33, 1])
@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("new,past,window", [
    ([1], [0], 0), ([1], [127], 0), ([1], [128], 0), ([2], [255], 0), ([3], [0], 0), ([130], [0], 0),
    ([1], [5000], 0), ([1], [5000], 128), ([5], [700], 100), ([40], [0], 1), ([300], [0], 128), ([65], [64], 257)])
def test_one_request(heads, f32, new, past, window):
    _check_all(new, past, heads, window, f32, seed=heads)


@pytest.mark.parametrize("heads", [64, 16, 5, 100, 128])
@pytest.mark.parametrize("window", [0, 128, 37])
@pytest.mark.parametrize("f32", [False, True])
def test_packed_requests(heads, window, f32):
    _check_all([1, 0, 70, 1, 1, 200, 0, 3, 1], [900, 40, 0, 0, 2000, 5, 0, 127, 128], heads, window, f32, seed=heads,
               stride=640, extra_q=3, extra_k=9)


@pytest.mark.parametrize("heads", [64, 20])
def test_many_rows(heads):
    # more row tiles than the SMs share: whole row tiles, several to a CTA
    _check_all([700, 1, 333], [0, 50, 200], heads if heads == 64 else 64, 0, False, seed=3)
    _check_all([2500, 77], [0, 3], heads, 128, False, seed=4)


def test_queries_without_keys():
    # more queries than latents: the first see nothing
    for heads in (64, 24):
        q, lat, *_, out, lse = _check_all([10, 4, 6], [-7, -4, 0], heads, 0, True, seed=heads)
        assert (out[:7] == 0).all() and (lse[:7] == -math.inf).all() and (lse[7:10] > -math.inf).all()
        assert (out[10:14] == 0).all()
        _check_all([10, 4], [-7, -4], heads, 3, False, seed=heads + 1)
    q = torch.randn(3, 8, 512, device="cuda").to(torch.bfloat16)       # no latent anywhere
    out, lse, err = _call(q, q.new_empty(0, 512), _cu([3]), _cu([0]))
    assert (out == 0).all() and (lse == -math.inf).all() and int(err) == 0


def test_sharp_and_flat_weights():
    # rising scores move the reference in every key tile; a huge one takes all
    csa2 = _csa2()
    n, heads = 900, 64
    q, lat = _inputs(5, [4], [n], heads)
    up = lat.clone()
    up *= torch.linspace(0.1, 12, n, device="cuda").to(torch.bfloat16)[:, None]
    cu_q, cu_k = _cu([4]), _cu([n])
    for x in (up, up.flip(0).contiguous(), torch.zeros_like(up)):
        for f32 in (False, True):
            out, lse, _ = _call(q, x, cu_q, cu_k, 0, f32)
            _check(out, lse, _ref(q, x, n - 4, 0))
    for scale in (0.0, -SCALE, 2.0):
        out, lse, _ = _call(q, lat, cu_q, cu_k, 0, True, scale=scale)
        _check(out, lse, _ref(q, lat, n - 4, 0, scale))
    # few keys need next to no workspace, many rows neither
    many = csa2.csa2_prompt_workspace_bytes(4, 64, 100000)
    assert max(csa2.csa2_prompt_workspace_bytes(4, 64, 128), csa2.csa2_prompt_workspace_bytes(5000, 64, 100000)) < many


@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("heads,window", [(64, 0), (16, 0), (16, 40), (100, 0), (64, 40), (64, 128), (128, 7), (64, 1)])
def test_latents_that_are_not_finite_reach_only_the_queries_that_see_them(value, heads, window):
    new, past = [30, 50, 3], [10, 0, 200]
    kv = [n + p for n, p in zip(new, past)]
    q, lat = _inputs(heads, new, kv, heads, 0, 60)
    cu_q, cu_k = _cu(new), _cu(kv)
    clean, clean_lse, _ = _call(q, lat, cu_q, cu_k, window)
    bad = lat.clone()
    at = 40 + 20                               # the second request's latent 20
    bad[at, 77] = value
    bad[sum(kv):] = value                      # rows behind the last request
    out, lse, _ = _call(q, bad, cu_q, cu_k, window)
    sees = torch.zeros(sum(new), dtype=torch.bool, device="cuda")
    sees[30 + 20:30 + 50 if not window else min(30 + 50, 30 + 20 + window)] = True
    assert torch.equal(out[~sees], clean[~sees]) and torch.equal(lse[~sees], clean_lse[~sees])
    if math.isnan(value):
        assert out[sees].isnan().all() and lse[sees].isnan().all()
    else:
        assert (~out[sees].isfinite()).any(-1).all()


@pytest.mark.parametrize("heads", [64, 128])
@pytest.mark.parametrize("window", [128, 127, 33, 1])
def test_windows_that_slide(heads, window):
    # long runs, requests that start anew, continue, have one token, or fewer latents than queries
    _check_all([400, 1, 1, 290, 5, 129, 700, 0, 128], [0, 0, 500, 31, -3, -129, 128, 9, 1], heads, window, False,
               seed=window)
    _check_all([3, 160], [1, 127], heads, window, True, seed=window)


@pytest.mark.parametrize("window", [128, 50])
def test_a_sliding_window_passes_over_latents_that_are_not_finite(window):
    n = 1500                                   # several tokens a run: bad ones ahead of it, inside it and behind it
    q, lat = _inputs(window, [n], [n], 64, 0, 4)
    clean, clean_lse, _ = _call(q, lat, _cu([n]), _cu([n]), window)
    bad = lat.clone()
    hit = torch.zeros(n, dtype=torch.bool, device="cuda")
    for at in (0, 3, 130, 700, 701, 1002, n - 1):
        bad[at] = float("nan")
        hit[at:at + window] = True
    bad[n:] = float("nan")
    out, lse, _ = _call(q, bad, _cu([n]), _cu([n]), window)
    assert torch.equal(out[~hit], clean[~hit]) and torch.equal(lse[~hit], clean_lse[~hit])
    assert out[hit].isnan().all() and lse[hit].isnan().all()


def test_queries_that_are_not_finite_stay_alone():
    q, lat = _inputs(9, [40], [40], 16)
    clean, _, _ = _call(q, lat, _cu([40]), _cu([40]))
    bad = q.clone()
    bad[8:16] = float("nan")                   # whole row tiles, and half of one
    bad[21, 3:9] = float("inf")
    out, _, _ = _call(bad, lat, _cu([40]), _cu([40]))
    hit = torch.zeros(40, 16, dtype=torch.bool, device="cuda")
    hit[8:16] = True
    hit[21, 3:9] = True
    assert torch.equal(out[~hit], clean[~hit]) and out[hit].isnan().all()


@pytest.mark.parametrize("heads", [64, 128])
@pytest.mark.parametrize("window", [128, 100, 1])
def test_queries_that_are_not_finite_leave_the_tokens_behind_them_alone(heads, window):
    # runs of tokens that share a ring of latents: every score of a key may be NaN though its latent is not
    n = 700
    q, lat = _inputs(heads + window, [n], [n], heads)
    clean, clean_lse, _ = _call(q, lat, _cu([n]), _cu([n]), window)
    bad = q.clone()
    hit = torch.zeros(n, heads, dtype=torch.bool, device="cuda")
    for t in (0, 3, 64, 250, 251, 600):
        bad[t, :64] = float("nan")
        hit[t, :64] = True
    out, lse, _ = _call(bad, lat, _cu([n]), _cu([n]), window)
    assert torch.equal(out[~hit], clean[~hit]) and torch.equal(lse[~hit], clean_lse[~hit])
    assert out[hit].isnan().all() and lse[hit].isnan().all()


def test_a_query_that_is_not_finite_over_shared_keys():
    q, lat = _inputs(11, [2], [9000], 64)      # every SM has a part of each token
    clean, clean_lse, _ = _call(q, lat, _cu([2]), _cu([9000]))
    bad = q.clone()
    bad[0] = float("nan")
    bad[1, 5] = float("nan")
    out, lse, _ = _call(bad, lat, _cu([2]), _cu([9000]))
    hit = bad.isnan().any(-1)
    assert torch.equal(out[~hit], clean[~hit]) and torch.equal(lse[~hit], clean_lse[~hit])
    assert out[hit].isnan().all() and lse[hit].isnan().all()


def test_bad_prefix_sums_are_reported():
    q, lat = _inputs(2, [100], [300], 24)
    i32 = dict(dtype=torch.int32, device="cuda")
    ok_q, ok_k = torch.tensor([0, 40, 100], **i32), torch.tensor([0, 100, 300], **i32)
    for cq, ck in (([0, 60, 40], None), ([5, 40, 100], None), ([0, 40, 101], None), ([0, -7, 100], None),
                   (None, [0, 400, 300]), (None, [0, 100, 10 ** 9]), (None, [-3, 100, 300]),
                   ([0, 2 ** 31 - 1, -2 ** 31], [2 ** 31 - 1, -2 ** 31, 2 ** 31 - 1])):
        _, _, err = _call(q, lat, ok_q if cq is None else torch.tensor(cq, **i32),
                          ok_k if ck is None else torch.tensor(ck, **i32))
        assert int(err) == 4


def test_repeats_are_identical_and_survive_capture_and_new_lengths():
    csa2 = _csa2()
    q, lat = _inputs(6, [64], [3000], 64)
    cu_q, cu_k = _cu([1] * 64), _cu([3000 // 64] * 63 + [3000 - 63 * (3000 // 64)])
    a = _call(q, lat, cu_q, cu_k)
    b = _call(q, lat, cu_q, cu_k)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    out, lse, err = torch.empty_like(a[0]), torch.empty_like(a[1]), torch.zeros_like(a[2])
    ws = torch.empty(csa2.csa2_prompt_workspace_bytes(64, 64, 3000), dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        csa2.csa2_prompt_attend(q, lat, cu_q, cu_k, 0, SCALE, out, lse, err, ws)
    g.replay()
    assert torch.equal(out, a[0]) and torch.equal(lse, a[1])
    # the captured call with other lengths: fewer tokens, other shares of the SMs
    new, kv = [1] * 20 + [0] * 44, [10, 2500] + [5] * 18 + [0] * 44
    cu_q.copy_(_cu(new))
    cu_k.copy_(_cu(kv))
    out.fill_(7)
    g.replay()
    ref = _call(q, lat, cu_q, cu_k)
    assert torch.equal(out, ref[0]) and (out[20:] == 7).all()
    _check(out[1:2], lse[1:2], _ref(q[1:2], lat[10:2510], 2499, 0))


def test_parts_join_through_the_log_sum_exp():
    # a prompt's past in two pieces, joined by csa2_combine as the sharded decode does
    csa2 = _csa2()
    n, heads = 1000, 64
    q, lat = _inputs(8, [3], [n], heads)
    parts = []
    for lo, hi in ((0, 400), (400, 997)):
        piece = lat[lo:hi].repeat(3, 1)
        parts.append(_call(q, piece, _cu([1, 1, 1]), _cu([hi - lo] * 3), f32=True))
    out = torch.empty(3, heads, 512, device="cuda")
    csa2.csa2_combine([p[0] for p in parts], [p[1] for p in parts], out)
    for t in range(3):
        o, l, mag, err = _ref(q[t:t + 1], lat[:997], 996, 0)
        assert ((out[t:t + 1].double() - o).abs() <= (2.0 ** -16 + 2 * err + 2.0 ** -18) * mag).all()


def test_padded_batch_leaves_the_rest_alone():
    # a captured batch's room with few live tokens, in every way of dealing the row tiles out
    for heads, window, live in ((64, 128, 37), (64, 0, 37), (20, 0, 900), (20, 100, 5), (64, 128, 0)):
        _check_all([live // 2, live - live // 2], [3, 0], heads, window, False, seed=live, extra_q=3000)


@pytest.mark.slow
def test_sizes_past_32_bits():
    # 66,001 tokens x 64 heads: more than 2^31 elements of q and of out
    n, heads = 66001, 64
    q = torch.randn(n, heads, 512, device="cuda", dtype=torch.bfloat16)
    lat = torch.randn(n, 512, device="cuda", dtype=torch.bfloat16)
    out, lse, err = _call(q, lat, _cu([n]), _cu([n]), 128)
    assert int(err) == 0
    for t in (0, 127, 128, 33000, n - 1):
        lo = max(0, t - 127)
        _check(out[t:t + 1], lse[t:t + 1], _ref(q[t:t + 1], lat[lo:t + 1], t - lo, 0), f"token {t}")
    del q, out
    # one token over 4,300,000 latents: 4.4 GB of them
    n = 4300000
    lat = torch.randn(n, 512, device="cuda", dtype=torch.bfloat16)
    q = torch.randn(1, 1, 512, device="cuda", dtype=torch.bfloat16) * 4
    out, lse, err = _call(q, lat, _cu([1]), _cu([n]), f32=True)
    assert int(err) == 0
    o, l, mag, e = _ref(q, lat, n - 1, 0)
    _check(out, lse, (o, l, mag, e))

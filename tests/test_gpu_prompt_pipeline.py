"""csa2_prompt_attend's pipeline of roles: what one row tile's output still needs is not overwritten by the row
tiles behind it, whatever else loads the memory."""
import pytest
import torch

from test_gpu_prompt import _call, _check, _cu, _inputs, _ref

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("heads,window", [(64, 128), (128, 100), (40, 200), (64, 0)])
def test_factors_last_until_the_output_has_used_them(heads, window, f32):
    # Two tokens of flat weights, then two of sharp ones, and so on: the sums that the rows are divided by differ
    # by up to a hundred times from one row tile to the next but one.  Copies on other streams hold back the stores.
    n = 1500
    q, lat = _inputs(heads, [n], [n], heads)
    q = q * torch.where(torch.arange(n, device="cuda") % 4 < 2, 0.0, 4.0).to(q.dtype)[:, None, None]
    cu = _cu([n])
    busy = [torch.empty(2, 1 << 27, dtype=torch.uint8, device="cuda") for _ in range(3)]
    streams = [torch.cuda.Stream() for _ in busy]
    torch.cuda.synchronize()
    runs = []
    for _ in range(6):
        for s, b in zip(streams, busy):
            with torch.cuda.stream(s):
                for _ in range(4):
                    b[0].copy_(b[1])
        runs.append(_call(q, lat, cu, cu, window, f32))
    torch.cuda.synchronize()
    for out, lse, err in runs:
        assert int(err) == 0 and torch.equal(out, runs[0][0]) and torch.equal(lse, runs[0][1])
    out, lse, _ = runs[0]
    for t in range(0, n, 250):
        lo = max(0, t + 1 - window) if window else 0
        _check(out[t:t + 250], lse[t:t + 250], _ref(q[t:t + 250], lat[lo:t + 250], t - lo, window), f"tokens from {t}")


@pytest.mark.parametrize("value", [float("inf"), -float("inf")])
@pytest.mark.parametrize("heads,new,past,window,f32", [
    (64, 700, 0, 128, False), (128, 300, 50, 100, False), (64, 300, 0, 0, False), (128, 100, 500, 0, True),
    (64, 2, 9000, 0, False), (64, 40, 9000, 0, True), (40, 200, 0, 0, False), (64, 200, 1000, 300, False)])
def test_infinite_queries_change_no_bit_of_the_others(value, heads, new, past, window, f32):
    # their scores are +inf or -inf, key by key: one is first without a reference and then far above it
    q, lat = _inputs(heads + new, [new], [new + past], heads)
    cu_q, cu_k = _cu([new]), _cu([new + past])
    clean, clean_lse, _ = _call(q, lat, cu_q, cu_k, window, f32)
    bad = q.clone()
    hit = torch.zeros(new, heads, dtype=torch.bool, device="cuda")
    for t in range(0, new, 3):
        for h in (t % heads, (7 * t + 1) % heads):
            bad[t, h, (t * 31 + h) % 512] = value
            hit[t, h] = True
    out, lse, err = _call(bad, lat, cu_q, cu_k, window, f32)
    assert int(err) == 0
    assert torch.equal(out[~hit], clean[~hit]) and torch.equal(lse[~hit], clean_lse[~hit])


@pytest.mark.parametrize("heads,new,past,window", [
    (64, [1000], [60000], 0), (64, [300], [60000], 0), (20, [3, 2900], [40000, 50000], 0), (64, [200], [70000], 65000),
    (128, [500, 1, 30], [1900, 50000, 40000], 0), (33, [800, 700], [2500, 9000], 5000), (64, [6000], [0], 0)])
def test_f32_outputs_over_many_latents(heads, new, past, window):
    # Latents of one sign, so that what the sums lose shows.  A score is off by err and a weight, in two bf16 parts,
    # by 2^-16; 16 key tiles of 16 products are added toward zero, each off by at most 2^-23 of a sum that grows
    # from nothing, half that of it all: 2^-16; fp32 additions of those sums over the past (500 at most) 2^-15 for the worst,
    # but their errors have either sign: 2^-19.
    kv = [n + p for n, p in zip(new, past)]
    q, lat = _inputs(heads, new, kv, heads)
    lat = lat.abs()
    q *= 0.5
    out, lse, err = _call(q, lat, _cu(new), _cu(kv), window, True)
    assert int(err) == 0
    a = c = 0
    for n, k in zip(new, kv):
        for t in sorted({0, n // 3, n - 1}):
            hi = k - n + t + 1
            lo = max(0, hi - window) if window else 0
            o, l, mag, e = _ref(q[a + t:a + t + 1], lat[c + lo:c + hi], hi - lo - 1, 0)
            got = out[a + t:a + t + 1].double()
            tol = (2 * 2.0 ** -16 + 2.0 ** -19 + 2 * e) * mag
            assert ((got - o).abs() <= tol).all(), float(((got - o).abs() / mag).max())
            # and in the mean, without the worst of every rounding
            assert float((got - o).norm() / o.norm()) < 1e-5
            assert ((lse[a + t:a + t + 1].double() - l).abs() <= e[..., 0] + 2.0 ** -20 * (1 + l.abs())).all()
        a, c = a + n, c + k

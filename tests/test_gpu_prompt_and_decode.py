"""What csa2_prompt_attend has to do with csa2_attend: the decode step's attention with every entry selected is the
window's and the entries', joined, not the dense one."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

U24 = 2.0 ** -24
SCALE = 1 / math.sqrt(512)


@pytest.mark.parametrize("n", [40, 300, 512])
@pytest.mark.parametrize("heads", [16, 64])
def test_decode_with_every_entry_selected_is_window_and_entries_joined(n, heads):
    import csa2_sparse_attention_decode_b200 as csa2
    from test_gpu_prompt import _call, _cu
    g = torch.Generator(device="cuda").manual_seed(n)
    # latents that FP4 and FP8 hold exactly: e2m1 values, with a 6 in every group of 16 channels
    values = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6], device="cuda")
    lat = values[torch.randint(0, 8, (n, 512), generator=g, device="cuda")]
    lat[:, ::16] = 6
    lat *= torch.randint(0, 2, (n, 512), generator=g, device="cuda") * 2 - 1
    cache = csa2.Cache(torch.arange(8, dtype=torch.int32, device="cuda")[None], 8, [1])
    csa2.csa2_prefill(cache, 0, 0, n, lat, torch.randn(n, 128, generator=g, device="cuda"), torch.zeros(n, device="cuda"))
    topk = torch.full((1, 512), -1, dtype=torch.int32, device="cuda")
    topk[0, :n] = torch.arange(n, device="cuda")
    q = (0.3 * torch.randn(n, heads, 512, generator=g, device="cuda")).to(torch.bfloat16)
    decode = torch.empty(1, heads, 512, device="cuda")
    csa2.csa2_attend(cache, q[-1:], topk, SCALE, decode, csa2.workspace(cache))
    assert csa2.csa2_get_device_error(cache) == 0

    lat16 = lat.to(torch.bfloat16)
    window, window_lse, _ = _call(q, lat16, _cu([n]), _cu([n]), csa2.SWA, True)
    dense, dense_lse, _ = _call(q, lat16, _cu([n]), _cu([n]), 0, True)
    joined = torch.empty(n, heads, 512, device="cuda")
    csa2.csa2_combine([window, dense], [window_lse, dense_lse], joined)

    keys = torch.cat([lat, lat[-128:]]).double()
    s = q[-1].double() @ keys.T * SCALE
    w = torch.softmax(s, -1)
    ref, mag = w @ keys, w @ keys.abs()
    # weights in two bf16 parts (2^-16), scores in fp32, the join (2^-18)
    err = 512 * U24 * SCALE * (q[-1].double().abs() @ keys.abs().T).amax(-1, keepdim=True)
    tol = (2.0 ** -16 + 2 * err + 2.0 ** -18) * mag
    assert ((decode[0].double() - ref).abs() <= tol).all()
    assert ((joined[-1].double() - ref).abs() <= tol).all()
    if n > 128:                                # where the window is not everything, dense attention is another answer
        assert not ((dense[-1].double() - ref).abs() <= tol).all()

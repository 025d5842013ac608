"""The workspace of csa2_prompt_attend: what its size is for one shape, and the bound for all."""
import os
import re

import pytest
import torch

import csa2_sparse_attention_decode_b200 as csa2

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_one_bound_holds_for_every_shape():
    with open(os.path.join(ROOT, "include", "csa2.h")) as f:
        said = re.search(r"CSA2_PROMPT_WORKSPACE_MAX \(\(size_t\)(\d+)\)", f.read())
    assert int(said.group(1)) == csa2.PROMPT_WORKSPACE_MAX
    sizes = [csa2.csa2_prompt_workspace_bytes(n_q, heads, n_k)
             for heads in (1, 8, 33, 64, 128) for n_q in (1, 2, 7, 32, 500, 896, 897, 5000, 1 << 20)
             for n_k in (0, 1, 128, 1280, 1281, 131072, 1 << 22, 2 ** 31 - 200)]
    assert 0 < min(sizes) and max(sizes) == csa2.PROMPT_WORKSPACE_MAX
    # not the largest shape's: a smaller one may need more
    assert csa2.csa2_prompt_workspace_bytes(100000, 64, 100000) < csa2.csa2_prompt_workspace_bytes(1, 64, 100000)


@pytest.mark.gpu
def test_one_workspace_serves_calls_of_every_shape():
    from test_gpu_prompt import _call, _check, _cu, _inputs, _ref
    ws = torch.empty(csa2.PROMPT_WORKSPACE_MAX, dtype=torch.uint8, device="cuda")
    for new, kv, heads, window in ((600, 600, 64, 0), (1, 5000, 64, 0), (3, 3000, 20, 0), (600, 600, 64, 128), (1, 1, 1, 0)):
        q, lat = _inputs(new, [new], [kv], heads)
        out, lse, err = _call(q, lat, _cu([new]), _cu([kv]), window, ws=ws)
        assert int(err) == 0
        for t in range(0, new, 200):
            lo = max(0, kv - new + t + 1 - window) if window else 0
            e = min(new, t + 200)
            _check(out[t:e], lse[t:e], _ref(q[t:e], lat[lo:kv - new + e], kv - new + t - lo, window))

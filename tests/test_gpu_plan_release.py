"""csa2_plan_tokens where pages come back."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu


def _i32(x):
    return torch.as_tensor(np.asarray(x, np.int32), device="cuda")


@pytest.mark.parametrize("B", [1, 3, 300])
def test_more_released_pages_than_the_stack_has_room_for(B):
    # pages held by a request and on the stack at once: the first ones go on it, and no word behind it is written
    import csa2_sparse_attention_decode_b200 as csa2
    held, n_pages = 4, 4 * B
    table = np.arange(n_pages, dtype=np.int32).reshape(B, held)
    room = n_pages - 3                         # of which all but three released ones find none
    free = np.arange(100, 100 + n_pages, dtype=np.int32) % n_pages
    whole = _i32(np.concatenate([free, [-77] * 8]))
    n_out, cu, err = _i32([-1]), _i32(np.full(B + 1, -1)), _i32([0])
    none = _i32([])
    csa2.csa2_plan_tokens(_i32([64 * held] * B), _i32([-64 * held] * B), _i32([1] * B), _i32(table), whole[:n_pages],
                          _i32([room]), n_out, cu, none, none, none, err)
    got = whole.cpu().numpy()
    assert got[:room].tolist() == free[:room].tolist() and got[room:n_pages].tolist() == [0, 1, 2]
    assert (got[n_pages:] == -77).all() and int(n_out) == n_pages and int(err) == 2 and not cu.any()

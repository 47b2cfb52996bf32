"""The 4-bit KV cache (pk_quant_*) at its limits: weights next to zero, values and
queries of very unequal size, refused steps, recorded failures."""
import math

import numpy as np
import pytest
import torch

from tests import quant_ref as ref
from tests.test_quant_cache import make_cache, make_rows, pk  # noqa: F401

gpu = pytest.mark.gpu
D, KEYS, BLOCK = 128, 32, 4608


# ---------------------------------------------------------------- eviction
@gpu
@pytest.mark.parametrize("lists", ["keep", "acc", "both", "none"])
@pytest.mark.parametrize("bh,n", [(3, 9000), (1, 20000), (40, 17003), (20, 40007), (2, 131075), (3, 290001)])
@pytest.mark.parametrize("zeros", [500, 3])
def test_evict_threshold_below_zero(pk, bh, n, zeros, lists):  # noqa: F811
    """The threshold is the largest negative weight, next to zeros of both signs (which share no digit with it), in
    few slots: the kept rows are the reference's, and nothing behind a pair's list or rows is written."""
    heavy, tied, budget = 1000, 2000, 2000
    cap = -(-n // KEYS) * KEYS
    rng = np.random.default_rng(n + zeros)
    acc = np.full((bh, cap), -1.0, np.float32)
    for p in range(bh):
        at = rng.permutation(n)
        acc[p, at[:heavy]] = 0.5
        acc[p, at[heavy:heavy + zeros]] = 0.0
        acc[p, at[heavy:heavy + zeros // 2]] = -0.0
        acc[p, at[heavy + zeros:heavy + zeros + tied]] = np.float32(-1e-45)
    g = torch.Generator(device="cuda").manual_seed(n)
    blocks = torch.randint(0, 256, (bh, cap // KEYS, BLOCK), generator=g, device="cuda", dtype=torch.uint8)
    lens = torch.full((bh,), n, dtype=torch.int32, device="cuda")
    src = pk.pk_quant_view(blocks, lens, pk.PK_BF16, acc=torch.from_numpy(acc).cuda())
    room = 64 * KEYS                     # 2048 slots: 48 behind the kept ones
    fill = torch.full((bh, 64, BLOCK), 0xA5, dtype=torch.uint8, device="cuda")
    dacc = torch.full((bh, room), 3.0, device="cuda") if lists in ("acc", "both") else None
    dst = pk.pk_quant_view(fill.clone(), torch.zeros(bh, dtype=torch.int32, device="cuda"), pk.PK_BF16, acc=dacc)
    store = torch.full((bh * budget + 2 * budget,), -7, dtype=torch.int32, device="cuda")
    keep = store[budget:-budget].view(bh, budget) if lists in ("keep", "both") else None
    pk.pk_quant_evict(src, dst, budget, keep=keep)
    assert dst.tensors[1].tolist() == [budget] * bh
    assert store[:budget].eq(-7).all() and store[-budget:].eq(-7).all()
    for p in range(bh):
        want = torch.from_numpy(ref.evict(acc[p], n, budget, 0, 0)).cuda()
        if keep is not None:
            assert torch.equal(keep[p].long(), want)
        if dacc is not None:
            assert torch.equal(dacc[p, :budget], src.tensors[2][p, want]) and dacc[p, budget:].eq(3.0).all()
        a, b = (x[p, :, 4096:].reshape(-1, 2, KEYS, 8).transpose(1, 2).reshape(-1, 16) for x in (blocks, dst.tensors[0]))
        assert torch.equal(a[want], b[:budget]) and b[budget:].eq(0xA5).all()          # scales
        a, b = (x[p, :, :2048].reshape(-1, 64) for x in (blocks, dst.tensors[0]))
        assert torch.equal(a[want], b[:budget]) and b[budget:].eq(0xA5).all()          # codes of K

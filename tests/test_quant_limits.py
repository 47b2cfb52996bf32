"""The 4-bit KV cache (pk_quant_*) at its limits: weights next to zero, values and
queries of very unequal size, refused steps, recorded failures."""
import math

import numpy as np
import pytest
import torch

from tests import quant_bound as bound
from tests import quant_ref as ref
from tests.test_quant_cache import make_cache, make_rows, pk  # noqa: F401

gpu = pytest.mark.gpu
D, KEYS, BLOCK = 128, 32, 4608


# ---------------------------------------------------------------- accuracy of the attention
def uneven(rng, G, n, td, ratio, where):
    """A query whose channel 5 of 128 is `ratio` times the others; in the keys that channel is nothing ("zero"), its
    group is ("group"), or its group is `ratio` times smaller than the others ("small")."""
    q = make_rows(rng, G, torch.float32).numpy()
    K, V = make_rows(rng, n, torch.float32).numpy(), make_rows(rng, n, torch.float32).numpy()
    q[:, 5] = np.abs(q).max() * ratio
    if where == "zero":
        K[:, 5] = 0
    elif where == "group":
        K[:, :32] = 0
    else:
        K[:, :32] /= ratio
    return torch.from_numpy(q).to(td), K, V


def check_close(pk, q, kinds, rows, accumulate=True, scale=None):  # noqa: F811
    """pk_quant_attend of q [bh][G][128] over pairs of rows (K, V) against 64 bits, within the bound of its arithmetic."""
    bh, G = q.shape[:2]
    lens = [len(K) for K, _ in rows]
    cap = max(KEYS, -(-max(lens) // KEYS) * KEYS)
    blocks = np.full((bh, cap // KEYS, BLOCK), 0xff, np.uint8)
    for p, (K, V) in enumerate(rows):
        if lens[p]:
            b = ref.pack(K, V)
            blocks[p, :len(b)] = b
    c = pk.pk_quant_view(torch.from_numpy(blocks).cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda"), kinds,
                         acc=torch.zeros(bh, cap, device="cuda"))
    out, lse = torch.zeros(bh, G, D, device="cuda"), torch.zeros(bh, G, device="cuda")
    work = torch.empty(pk.pk_quant_attend_workspace(c, G, accumulate), dtype=torch.uint8, device="cuda")
    pk.pk_quant_attend(c, q.cuda(), G, out, work, lse=lse, accumulate=accumulate, scale=scale or 0.0)
    out, lse, acc = (t.cpu().double().numpy() for t in (out, lse, c.tensors[2]))
    for p, n in enumerate(lens):
        if n == 0:
            assert np.all(out[p] == 0) and np.all(lse[p] == -np.inf)
            continue
        K, V = (x[:n] for x in ref.values(blocks[p]))
        o, l, w, eo, el, ew = bound.attend(q[p].double().numpy(), K, V, scale)
        assert np.all(np.abs(out[p] - o) <= eo), (p, n, np.max(np.abs(out[p] - o) / eo))
        assert np.all(np.abs(lse[p] - l) <= el), (p, n, np.max(np.abs(lse[p] - l) / el))
        if accumulate:                   # each weight's own error, a rounding a head
            tol = (w * ew).sum(0) + (G + 1) * bound.U * w.sum(0) + 1e-37
            assert np.all(np.abs(acc[p, :n] - w.sum(0)) <= tol), (p, n, np.max(np.abs(acc[p, :n] - w.sum(0)) / tol))


@pytest.mark.parametrize("n", [2, 5, 33, 577])
@pytest.mark.parametrize("form", ["q 15 bits", "weights as halves", "logits as halves"])
def test_bound_tells_coarser_forms(n, form):
    """What fewer bits would do is outside of the bound, and q as it is held well inside.  (From two keys on: a single
    key's weight is 1, and 1 times a scale of 8 bits is a half.)"""
    rng = np.random.default_rng(n)
    q = (1.5 * make_rows(rng, 8, torch.float32)).double().numpy()
    K, V = (ref.stored(make_rows(rng, n, torch.float32).numpy())[2] for _ in range(2))
    o, l, _, eo, el, _ = bound.attend(q, K, V)
    go, gl = bound.coarse(q, K, V, form)
    assert np.any(np.abs(go - o) > eo) or np.any(np.abs(gl - l) > el)
    fo, fl = bound.coarse(bound.fixed_point(q), K, V, "")
    assert np.all(np.abs(fo - o) <= 0.5 * eo) and np.all(np.abs(fl - l) <= 0.5 * el)


@pytest.mark.parametrize("form,where,ratio", [
    ("q 22 bits of all", "zero", 1024), ("q 22 bits of all", "small", 1024), ("q 22 bits of all", "group", 256),
    ("q 30 bits of all", "group", 2 ** 18), ("q 30 bits of all", "small", 2 ** 18),
])
def test_bound_tells_a_unit_for_all_channels(form, where, ratio):
    """A unit for the head's largest channel, beside small ones that decide."""
    rng = np.random.default_rng(ratio)
    q, K, V = uneven(rng, 4, 200, torch.float32, ratio, where)
    q = q.double().numpy()
    K, V = ref.stored(K)[2], ref.stored(V)[2]
    o, l, _, eo, el, _ = bound.attend(q, K, V)
    go, gl = bound.coarse(q, K, V, form)
    assert np.any(np.abs(go - o) > eo) and np.any(np.abs(gl - l) > el)


@gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("G", [1, 4, 5, 8])
@pytest.mark.parametrize("where", ["zero", "group", "small"])
def test_attend_query_of_uneven_channels(pk, G, dtype, where):  # noqa: F811
    """A channel of q far above the others that the keys hardly have: the others decide, as accurately as ever."""
    td, kind = (torch.bfloat16, pk.PK_BF16) if dtype == "bf16" else (torch.float32, pk.PK_F32)
    rng = np.random.default_rng(G)
    parts = [uneven(rng, G, n, td, ratio, where) for n in (1, 33, 500) for ratio in (16, 256, 1024, 16384, 2 ** 20)]
    check_close(pk, torch.stack([x[0] for x in parts]), kind, [x[1:] for x in parts])


@gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("G", [1, 3, 4, 5, 8])
@pytest.mark.parametrize("lens", [[1, 2, 3, 31, 32, 33, 0, 64, 100, 577], [1000, 9001], [20011], [65] * 140, [33, 700] * 20])
def test_attend_within_the_bound_of_its_arithmetic(pk, G, dtype, lens):  # noqa: F811
    td, kind = (torch.bfloat16, pk.PK_BF16) if dtype == "bf16" else (torch.float32, pk.PK_F32)
    rng = np.random.default_rng(len(lens) + G)
    q = torch.stack([(1.5 * make_rows(rng, G, torch.float32)).to(td) for _ in lens])
    rows = [tuple(make_rows(rng, n, td).float().numpy() for _ in range(2)) for n in lens]
    check_close(pk, q, kind, rows)
    check_close(pk, q, kind, rows, accumulate=False, scale=0.011)


@gpu
@pytest.mark.parametrize("G", [3, 4, 5, 8])
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_attend_poisoned_query_head(pk, G, bad):  # noqa: F811
    """A NaN or an infinity in one head's query makes that head NaN, of every pair length, and no other."""
    rng = np.random.default_rng(G)
    lens = [1, 32, 33, 700]
    c, blocks = make_cache(pk, rng, lens, 704, pk.PK_F32)
    q = torch.stack([make_rows(rng, G, torch.float32) for _ in lens])
    for p in range(len(lens)):
        q[p, p % G, 37 * p % D] = bad
    out, lse = torch.zeros(len(lens), G, D, device="cuda"), torch.zeros(len(lens), G, device="cuda")
    pk.pk_quant_attend(c, q.cuda(), G, out, torch.empty(pk.pk_quant_attend_workspace(c, G), dtype=torch.uint8, device="cuda"), lse=lse)
    out, lse = out.cpu().double().numpy(), lse.cpu().double().numpy()
    for p, n in enumerate(lens):
        K, V = (x[:n] for x in ref.values(blocks[p]))
        ok = [g for g in range(G) if g != p % G]
        assert np.isnan(out[p, p % G]).all() and np.isnan(lse[p, p % G])
        o, l, _, eo, el, _ = bound.attend(q[p, ok].double().numpy(), K, V)
        assert np.all(np.abs(out[p, ok] - o) <= eo) and np.all(np.abs(lse[p, ok] - l) <= el)


def flat_logits(n, at, z):
    """Keys whose logit with q = 0.5 is z everywhere and 0 at the places `at`."""
    K = np.full((n, D), z * math.sqrt(D) / (0.5 * D), np.float32)
    K[at] = 0
    return K


@gpu
@pytest.mark.parametrize("G", [1, 8])
@pytest.mark.parametrize("size", [1e15, 1e21, 1e28])
def test_attend_small_weights_beside_huge_values(pk, G, size):  # noqa: F811
    """Keys of values up to 2^96: the others' weights count all the same, in the outputs, the log-sums and acc."""
    rng = np.random.default_rng(G)
    n = 20001
    V = make_rows(rng, n, torch.float32).numpy()
    rows = []
    for at in ([0], [n - 1], [7, 11111, n - 9]):                         # 9e-5 of a huge key's weight each, 2 in all
        v = V.copy()
        v[at] = size * np.sign(v[at])
        rows.append((flat_logits(n, at, -9.3), v))
    v = V.copy()
    v[14000:] = np.clip(v[14000:] * np.float32(size), -7e28, 7e28)       # huge from some place on
    rows.append((make_rows(rng, n, torch.float32).numpy(), v))
    v = V.copy()
    v[500] = size                                                        # nobody looks at it
    K = make_rows(rng, n, torch.float32).numpy()
    K[500] = -300
    rows.append((K, v))
    check_close(pk, torch.full((len(rows), G, D), 0.5), pk.PK_F32, rows)


@gpu
@pytest.mark.parametrize("G", [2, 6])
@pytest.mark.parametrize("size", [1.0, 1e6, 1e12, 7e28])
def test_attend_rows_of_zeros_beside_large_values(pk, G, size):  # noqa: F811
    """Keys whose values are zero, or next to it, take their share of the weights from keys of large ones."""
    n = 20001
    rows = []
    for at in ([0], [n - 1], [7, 11111, n - 9], list(range(0, n, 37))):  # 9e-5 of the others' weight each, 2 in all
        for small in (0.0, 1e-30):
            V = np.full((n, D), small, np.float32)
            V[at] = size
            rows.append((flat_logits(n, at, -9.3), V))
    check_close(pk, torch.full((len(rows), G, D), 0.5), pk.PK_F32, rows)


@gpu
@pytest.mark.parametrize("G", [2, 7])
def test_attend_values_small_then_huge(pk, G):  # noqa: F811
    """Values far below one, then a huge one without weight, then small ones again."""
    rng = np.random.default_rng(G)
    n = 20001
    K = make_rows(rng, n, torch.float32).numpy()
    rows = []
    for small in (1e-3, 1e-20):
        V = make_rows(rng, n, torch.float32, small).numpy()
        K = K.copy()
        K[9999] = -500
        V[9999] = 7e28
        rows.append((K, V))
    check_close(pk, torch.full((2, G, D), 0.5), pk.PK_F32, rows)


@gpu
@pytest.mark.parametrize("G", [4, 5])
def test_attend_huge_keys(pk, G):  # noqa: F811
    """Keys near the end of fp32's range and queries as small, of ordinary logits and of such that the largest takes all."""
    rng = np.random.default_rng(G)
    K, V = make_rows(rng, 300, torch.float32, 1e33).numpy(), make_rows(rng, 300, torch.float32).numpy()
    q = make_rows(rng, G, torch.float32, 1e-33)
    check_close(pk, q[None], pk.PK_F32, [(K, V)])
    q = make_rows(rng, G, torch.float32, 1e-29)
    blocks = torch.from_numpy(ref.pack(K, V)[None]).cuda()
    c = pk.pk_quant_view(blocks, torch.full((1,), 300, dtype=torch.int32, device="cuda"), pk.PK_F32)
    out = torch.zeros(1, G, D, device="cuda")
    pk.pk_quant_attend(c, q.cuda()[None], G, out, torch.empty(pk.pk_quant_attend_workspace(c, G), dtype=torch.uint8, device="cuda"))
    K, V = ref.values(blocks[0].cpu().numpy())
    top = (q.double().numpy() @ K[:300].T).argmax(1)
    # logits of about 1e4: the others' weights are below e^-30, together 300 e^-30, and not zero where V[top] is (head 3 of 5:
    # e^-84 for the next one); one weight, held as a pair of halves (2^-22), times one value
    assert np.allclose(out[0].cpu().double().numpy(), V[top], rtol=2.0 ** -20, atol=300 * math.exp(-30) * np.abs(V[:300]).max())


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


@gpu
@pytest.mark.parametrize("cap", [1024, 40032, 131104])
@pytest.mark.parametrize("budget,sink,recent", [(500, 5, 10), (30, 10, 20), (900, 0, 900), (1000, 1000, 0)])
def test_evict_of_bad_and_short_lengths(pk, cap, budget, sink, recent):  # noqa: F811
    """Lengths beyond the room or below zero are read as the bounds and recorded; pairs within the budget keep all; a
    budget that sink and recent use up; all in one call, whatever kernel the room asks for."""
    lens = [cap, 0, 1, budget, budget + 1, cap + 7, -3]
    use = [min(max(n, 0), cap) for n in lens]
    g = torch.Generator(device="cuda").manual_seed(cap + budget)
    blocks = torch.randint(0, 256, (len(lens), cap // KEYS, BLOCK), generator=g, device="cuda", dtype=torch.uint8)
    acc = torch.rand(len(lens), cap, generator=g, device="cuda")
    src = pk.pk_quant_view(blocks, torch.tensor(lens, dtype=torch.int32, device="cuda"), pk.PK_BF16, acc=acc,
                           status=torch.zeros(2, dtype=torch.int32, device="cuda"))
    dst = pk.pk_quant_view(torch.zeros(len(lens), 32, BLOCK, dtype=torch.uint8, device="cuda"),
                           torch.zeros(len(lens), dtype=torch.int32, device="cuda"), pk.PK_BF16)
    keep = torch.zeros(len(lens), budget, dtype=torch.int32, device="cuda")
    pk.pk_quant_evict(src, dst, budget, sink=sink, recent=recent, keep=keep)
    assert src.tensors[3][0].item() == pk._lib.PK_ERR_DEVICE_CHECK and src.tensors[3][1].item() in (5, 6)
    for p, n in enumerate(use):
        want = ref.evict(acc[p].cpu().numpy(), n, budget, sink, recent)
        assert dst.tensors[1][p].item() == len(want)
        assert keep[p].tolist() == want.tolist() + [-1] * (budget - len(want))
        rows = torch.from_numpy(want).cuda()
        a, b = (x[p, :, :2048].reshape(-1, 64) for x in (blocks, dst.tensors[0]))
        assert torch.equal(a[rows], b[:len(want)]) and b[len(want):].eq(0).all()


# ---------------------------------------------------------------- the bounded decode cache
def bad_steps(dev, dtype):
    """Arguments of a step of a cache of 1 x 2 pairs and 3 query heads, each with one that does not fit."""
    q, k = torch.zeros(1, 6, D, dtype=dtype, device=dev), torch.zeros(1, 2, 1, D, dtype=dtype, device=dev)
    other = torch.float32 if dtype == torch.bfloat16 else torch.bfloat16
    return [(q[:, :5], k, k), (q[0], k, k), (q.to(other), k, k), (q, k[:, :1], k), (q, k.to(other), k), (q, k, k.to(other)),
            (q, k, k[..., :64]), (q.to("meta"), k, k), (q, k.to("meta"), k), (q, k, k.to("meta"))]


def test_bounded_cache_checks_a_step_first(pk):  # noqa: F811
    """A step's arguments are checked before its first call (which has no GPU to run on here)."""
    from kv_cache_top_b200.bounded_cache import BoundedCache
    K = torch.zeros(1, 2, 0, D)
    c = BoundedCache(K, K, group=3, budget=8, sink=0, recent=0)
    for args in bad_steps("cpu", torch.float32):
        with pytest.raises(ValueError):
            c.step(*args)
        assert (c.n, c.T, c.evictions) == (0, 0, 0)
    for scale in (-1.0, math.nan, math.inf):
        with pytest.raises(ValueError):
            BoundedCache(K, K, group=3, budget=8, sink=0, recent=0, scale=scale)


@gpu
def test_bounded_cache_refused_step_changes_nothing(pk):  # noqa: F811
    """Full or not, a refused step neither evicts nor adds; the corrected one goes on as if it had not been."""
    from kv_cache_top_b200.bounded_cache import BoundedCache
    rng = np.random.default_rng(2)
    K, V = (make_rows(rng, 2 * 5, torch.bfloat16).view(1, 2, 5, D).cuda() for _ in range(2))
    a, b = (BoundedCache(K, V, group=3, budget=6, sink=1, recent=2, update=2) for _ in range(2))
    for _ in range(7):
        q = make_rows(rng, 6, torch.bfloat16).view(1, 6, D).cuda()
        k, v = (make_rows(rng, 2, torch.bfloat16).view(1, 2, 1, D).cuda() for _ in range(2))
        before = [x.clone() for x in (a.positions, a.weights, *a.rows(), a._cache.tensors[1])] + [a.n, a.T, a.evictions]
        for args in bad_steps("cuda", torch.bfloat16) + [(q.cpu(), k, v), (q, k.cpu(), v), (q, k, v.cpu())]:
            with pytest.raises(ValueError):
                a.step(*args)
        after = [a.positions, a.weights, *a.rows(), a._cache.tensors[1], a.n, a.T, a.evictions]
        assert all(torch.equal(x, y) if isinstance(x, torch.Tensor) else x == y for x, y in zip(before, after))
        assert torch.equal(a.step(q, k, v), b.step(q, k, v))
        assert torch.equal(a.positions, b.positions) and torch.equal(a.weights, b.weights)
    assert a.evictions == b.evictions >= 2


def test_bounded_cache_check_reads_the_status(pk):  # noqa: F811
    """Both buffers share one status word; check() raises what it holds, once."""
    from kv_cache_top_b200.bounded_cache import BoundedCache
    K = torch.zeros(1, 2, 0, D)
    c = BoundedCache(K, K, group=3, budget=8, sink=0, recent=0)
    c.check()
    other, _ = c._buffers(8)
    for status, pair in ((pk._lib.PK_ERR_DEVICE_CHECK, 1), (pk._lib.PK_ERR_TIMEOUT, 0)):
        other.tensors[3].copy_(torch.tensor([status, pair], dtype=torch.int32))
        with pytest.raises(pk.PkError) as e:
            c.check()
        assert e.value.status == status and "pair %d" % pair in str(e.value)
        c.check()


@gpu
def test_bounded_cache_check_raises_what_the_kernels_recorded(pk):  # noqa: F811
    """A length out of range, found before or after an eviction gave up the prompt's buffer; without one check() passes."""
    from kv_cache_top_b200.bounded_cache import BoundedCache
    rng = np.random.default_rng(3)
    K, V = (make_rows(rng, 2 * 200, torch.float32).view(1, 2, 200, D).cuda() for _ in range(2))
    new = [make_rows(rng, 2, torch.float32).view(1, 2, 1, D).cuda() for _ in range(2)]
    q = make_rows(rng, 6, torch.float32).view(1, 6, D).cuda()
    for when in ("never", "before", "after"):
        c = BoundedCache(K, V, group=3, budget=40, sink=1, recent=20, update=8)
        if when == "before":
            c._cache.tensors[1][1] = -5
            c.observe(q)
            c._cache.tensors[1][1] = 200
        c.step(q, *new)                  # evicts from the prompt's buffer
        assert c.evictions == 1 and c.n == 41
        if when == "after":
            c._cache.tensors[1][1] = c._cache.n_cap + 1
            c.observe(q)
        if when == "never":
            c.check()
        else:
            with pytest.raises(pk.PkError) as e:
                c.check()
            assert e.value.status == pk._lib.PK_ERR_DEVICE_CHECK and "pair 1" in str(e.value)
        c.check()


@gpu
def test_bounded_cache_gives_up_a_long_prompt(pk):  # noqa: F811
    """After the eviction of a long prompt the cache holds what its bound needs: blocks, positions and workspace."""
    from kv_cache_top_b200.bounded_cache import BoundedCache
    T0 = 30000
    torch.cuda.synchronize()
    before = torch.cuda.memory_allocated()
    K = torch.zeros(1, 2, T0, D, dtype=torch.bfloat16, device="cuda")
    c = BoundedCache(K, K, group=4, budget=64, sink=1, recent=20, update=64)
    q, k = torch.zeros(1, 8, D, dtype=torch.bfloat16, device="cuda"), torch.zeros(1, 2, 1, D, dtype=torch.bfloat16, device="cuda")
    del K
    for _ in range(130):                 # past the second eviction
        c.step(q, k, k)
    c.check()
    assert c.evictions == 3
    small = pk.pk_quant_attend_workspace(c._cache, 4, True)
    assert c._work.numel() == small
    # two buffers of 128 keys (144 bytes, a weight, a position), outputs, the list, the arguments; torch rounds up to 512
    room = small + 2 * 2 * 128 * (144 + 4 + 8) + 32 * 1024
    torch.cuda.synchronize()
    assert torch.cuda.memory_allocated() - before <= room < T0 * 2 * 144

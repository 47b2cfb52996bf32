"""The 4-bit KV cache (pk_quant_*): rows in and out, attention over the cache,
eviction by accumulated weight, each against a plain 64-bit implementation of
the documented format (tests/quant_ref.py)."""
import ctypes as C
import math

import numpy as np
import pytest
import torch

from tests import quant_ref as ref

gpu = pytest.mark.gpu
D, KEYS, BLOCK = 128, 32, 4608


@pytest.fixture(scope="module")
def pk():
    from kv_cache_top_b200 import build
    build.build()
    import kv_cache_top_b200 as pk
    return pk


def dt(pk, name):
    return (torch.bfloat16, pk.PK_BF16) if name == "bf16" else (torch.float32, pk.PK_F32)


def make_rows(rng, n, dtype, scale=1.0):
    spread = np.exp(0.5 * rng.standard_normal(D))
    return torch.from_numpy((rng.standard_normal((n, D)) * spread * scale).astype(np.float32)).to(dtype)


def make_cache(pk, rng, lens, cap, kind, acc=None, status=True, v_scale=1.0):
    """A cache on the GPU of the given lengths; rows behind a length are 0xff bytes."""
    bh = len(lens)
    blocks = np.full((bh, cap // KEYS, BLOCK), 0xff, np.uint8)
    dtype = torch.bfloat16 if kind == pk.PK_BF16 else torch.float32
    for p, n in enumerate(lens):
        if n:
            b = ref.pack(make_rows(rng, n, dtype).float().numpy(), make_rows(rng, n, dtype, v_scale).float().numpy())
            blocks[p, :len(b)] = b
    t = torch.from_numpy(blocks).cuda()
    st = torch.zeros(2, dtype=torch.int32, device="cuda") if status else None
    a = None if acc is None else torch.from_numpy(acc.astype(np.float32)).cuda()
    return pk.pk_quant_view(t, torch.tensor(lens, dtype=torch.int32, device="cuda"), kind, acc=a, status=st), blocks


# ---------------------------------------------------------------- on the CPU
def test_reference_format_round_trip():
    """The test's packing and decoding agree with each other and with the documented bound."""
    rng = np.random.default_rng(0)
    K, V = (make_rows(rng, 45, torch.float32).numpy() for _ in range(2))
    b = ref.pack(K, V)
    k, v = ref.values(b)
    for x, y in ((K, k), (V, v)):
        assert np.array_equal(y[:45], ref.stored(x)[2])
        s = ref.stored(x)[1][:, ref.GROUP]
        assert np.all(np.abs(x - y[:45]) <= s * (0.5 + 7 * 2.0 ** -8))     # half a step, and the scale's rounding
    assert sorted(ref.K_NIB) == list(range(D)) and all(sorted(v) == list(range(D)) for v in ref.V_NIB)


def test_refusals_before_any_launch(pk):
    lib, L = pk.lib, pk._lib
    fake = 1 << 20                       # never dereferenced: sizes are checked first, then the pointers
    one = C.c_size_t()

    def view(bh=2, kind=1, cap=64, blocks=fake, lens=fake, acc=None, status=None):
        return pk.pk_quant_cache(bh, kind, cap, blocks, lens, acc, status)

    size = lambda c, g=4, a=0: lib.pk_quant_attend_workspace(c, g, a, C.byref(one))  # noqa: E731
    assert size(view()) == L.PK_OK and one.value > 0 and one.value % 256 == 0
    small = one.value
    assert size(view(), 4, 1) == L.PK_OK and one.value == small + 2 * 4 * 64 * 4
    assert size(None) == L.PK_ERR_INVALID_ARG
    for bad in (view(bh=0), view(kind=2), view(cap=0), view(cap=33), view(cap=-32)):
        assert size(bad) == L.PK_ERR_INVALID_ARG
    assert size(view(bh=65536)) == L.PK_ERR_UNSUPPORTED
    assert size(view(cap=1 << 31)) == L.PK_ERR_CAPACITY
    assert size(view(), 0) == L.PK_ERR_INVALID_ARG and size(view(), 9) == L.PK_ERR_INVALID_ARG
    assert lib.pk_quant_attend_workspace(view(), 4, 0, None) == L.PK_ERR_INVALID_ARG
    # without a GPU no pointer is device memory: every launching call refuses
    assert lib.pk_quant_append(None, None, None, 1, 0, None, None) == L.PK_ERR_INVALID_ARG
    assert lib.pk_quant_append(view(blocks=None), fake, fake, 1, 0, None, None) == L.PK_ERR_INVALID_ARG
    assert lib.pk_quant_rows(view(lens=None), 1, fake, fake, None, None) == L.PK_ERR_INVALID_ARG
    assert lib.pk_quant_attend(view(), None, 4, 0.0, None, None, 0, None, 0, None) == L.PK_ERR_INVALID_ARG
    assert lib.pk_quant_evict(view(), None, 1, 0, 0, None, None) == L.PK_ERR_INVALID_ARG


def test_view_checks_tensors(pk):
    blocks, lens = torch.zeros(2, 3, BLOCK, dtype=torch.uint8), torch.zeros(2, dtype=torch.int32)
    c = pk.pk_quant_view(blocks, lens, pk.PK_BF16)
    assert (c.bh, c.n_cap, c.kv_dtype) == (2, 96, pk.PK_BF16) and c.blocks == blocks.data_ptr() and not c.acc
    for bad in (dict(blocks=blocks[:, :, :100]), dict(blocks=blocks.to(torch.int8)), dict(lens=lens.long()),
                dict(lens=torch.zeros(3, dtype=torch.int32)), dict(acc=torch.zeros(2, 64)),
                dict(acc=torch.zeros(2, 96, dtype=torch.float64)), dict(status=torch.zeros(1, dtype=torch.int32)),
                dict(blocks=torch.zeros(2, 6, BLOCK, dtype=torch.uint8)[:, ::2])):
        with pytest.raises(ValueError):
            pk.pk_quant_view(**{**dict(blocks=blocks, lens=lens, kv_dtype=pk.PK_BF16), **bad})


# ---------------------------------------------------------------- refusals with real pointers
@gpu
def test_gpu_refusals(pk):
    rng = np.random.default_rng(1)
    c, _ = make_cache(pk, rng, [3, 40], 64, pk.PK_BF16, acc=np.zeros((2, 64)))
    plain, _ = make_cache(pk, rng, [3, 40], 64, pk.PK_BF16)
    k = torch.zeros(2, 4, D, dtype=torch.bfloat16, device="cuda")
    out = torch.zeros(2, 4, D, device="cuda")
    work = torch.empty(pk.pk_quant_attend_workspace(c, 4, True), dtype=torch.uint8, device="cuda")

    def refused(status, f, *args, **kw):
        with pytest.raises(pk.PkError) as e:
            f(*args, **kw)
        assert e.value.status == status, (f, e.value.status)

    bad, cap = pk._lib.PK_ERR_INVALID_ARG, pk._lib.PK_ERR_CAPACITY
    refused(bad, pk.pk_quant_append, c, k, k, 0)
    refused(cap, pk.pk_quant_append, c, k, k, 65)
    refused(bad, pk.pk_quant_append, c, k, k, 4, src_stride=3)
    refused(bad, pk.pk_quant_append, c, k.cpu(), k, 4)
    refused(bad, pk.pk_quant_append, c, k.data_ptr() + 1, k, 4)
    refused(bad, pk.pk_quant_append, c, k, k, 4, at=torch.zeros(2, dtype=torch.int32))
    refused(bad, pk.pk_quant_rows, c, 0, k, k)
    refused(bad, pk.pk_quant_rows, c, 1, None, k)
    refused(bad, pk.pk_quant_attend, c, k, 0, out, work)
    refused(bad, pk.pk_quant_attend, c, k, 9, out, work)
    refused(bad, pk.pk_quant_attend, c, k, 4, out, work, scale=-1.0)
    refused(bad, pk.pk_quant_attend, c, k, 4, out, work, scale=math.nan)
    refused(bad, pk.pk_quant_attend, c, k, 4, out, work, scale=math.inf)
    refused(bad, pk.pk_quant_attend, c, k, 4, out.data_ptr() + 2, work)
    refused(bad, pk.pk_quant_attend, plain, k, 4, out, work, accumulate=True)
    refused(bad, pk.pk_quant_attend, c, k, 4, out, work[8:])
    refused(cap, pk.pk_quant_attend, c, k, 4, out, work[:-256], accumulate=True)
    d, _ = make_cache(pk, rng, [0, 0], 32, pk.PK_BF16, acc=np.zeros((2, 32)))
    refused(bad, pk.pk_quant_evict, plain, d, 32)                    # no weights to go by
    refused(bad, pk.pk_quant_evict, c, d, 0)
    refused(bad, pk.pk_quant_evict, c, d, 32, sink=-1)
    refused(bad, pk.pk_quant_evict, c, d, 32, sink=20, recent=13)
    refused(cap, pk.pk_quant_evict, c, d, 33)
    refused(bad, pk.pk_quant_evict, c, c, 32)
    f32, _ = make_cache(pk, rng, [0, 0], 64, pk.PK_F32)
    refused(bad, pk.pk_quant_evict, c, f32, 32)
    few, _ = make_cache(pk, rng, [0], 64, pk.PK_BF16)
    refused(bad, pk.pk_quant_evict, c, few, 32)
    torch.cuda.synchronize()
    assert c.tensors[1].tolist() == [3, 40] and c.tensors[3].tolist() == [0, 0]


@gpu
def test_evict_list_in_a_cache_is_refused(pk):
    """keep is read while the caches are written: it lies outside of them."""
    rng = np.random.default_rng(15)
    c, _ = make_cache(pk, rng, [40, 64], 64, pk.PK_BF16, acc=np.ones((2, 64)))
    d, _ = make_cache(pk, rng, [0, 0], 32, pk.PK_BF16, acc=np.zeros((2, 32)))
    before = [t.clone() for t in (*c.tensors, *d.tensors)]
    for t in (*c.tensors[:3], *d.tensors[:3]):
        with pytest.raises(pk.PkError) as e:
            pk.pk_quant_evict(c, d, 32, keep=t.data_ptr())
        assert e.value.status == pk._lib.PK_ERR_INVALID_ARG
    torch.cuda.synchronize()
    assert all(torch.equal(x, t) for x, t in zip(before, (*c.tensors, *d.tensors)))


# ---------------------------------------------------------------- rows in and out
@gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("lens,n_new,stride,shift", [
    ([0], 1, 0, 0), ([31], 1, 0, 0), ([0, 5, 63], 1, 3, 1), ([0, 1, 30, 33], 64, 0, 0), ([7, 0], 65, 70, 1),
    ([2, 100], 333, 0, 2), ([0] * 5, 32, 0, 8),
])
def test_append_codes_are_exact(pk, dtype, lens, n_new, stride, shift):
    """Codes and scales of every new row are the reference's; other bytes of the cache do not change; lengths grow.
    `shift` elements off the 16-byte boundary."""
    td, kind = dt(pk, dtype)
    rng = np.random.default_rng(len(lens) * 1000 + n_new)
    cap = -(-(max(lens) + n_new) // KEYS) * KEYS + KEYS
    bh, st = len(lens), stride or n_new
    c, before = make_cache(pk, rng, lens, cap, kind, acc=rng.random((bh, cap)))
    acc0 = c.tensors[2].cpu().numpy()
    rows = []
    for _ in range(2):
        x = make_rows(rng, bh * st, td)
        x[::3, 5] *= 9
        x[1::4, 32:64] = 0
        x[::5, 96:] = x[::5, 96:].sign() * torch.tensor(rng.integers(0, 8, 32), dtype=td) * 0.5    # ties and borders
        flat = torch.zeros(x.numel() + shift, dtype=td, device="cuda")
        flat[shift:] = x.flatten().cuda()
        rows.append((x.view(bh, st, D), flat[shift:].view(bh, st, D)))
    pk.pk_quant_append(c, rows[0][1], rows[1][1], n_new, src_stride=stride)
    got = c.tensors[0].cpu().numpy()
    assert c.tensors[1].tolist() == [n + n_new for n in lens] and c.tensors[3].tolist() == [0, 0]
    for p, n in enumerate(lens):
        kc, vc, ks, vs = ref.decode(got[p])
        for code, s, x in ((kc, ks, rows[0][0]), (vc, vs, rows[1][0])):
            want, scale, _ = ref.stored(x[p, :n_new].float().numpy())
            assert np.array_equal(s[n:n + n_new], scale)
            assert np.array_equal(code[n:n + n_new], want)
        for a, b in zip(ref.decode(before[p]), (kc, vc, ks, vs)):
            keep = np.ones(cap, bool)
            keep[n:n + n_new] = False
            assert np.array_equal(a[keep], b[keep], equal_nan=True)
        acc = c.tensors[2][p].cpu().numpy()
        assert np.all(acc[n:n + n_new] == 0) and np.array_equal(acc[:n], acc0[p, :n]) and \
            np.array_equal(acc[n + n_new:], acc0[p, n + n_new:])


@gpu
def test_append_extreme_values(pk):
    """Subnormal, huge, infinite and NaN values; a group's neighbours are not touched by it."""
    rng = np.random.default_rng(5)
    x = rng.standard_normal((12, D)).astype(np.float32)
    x[0] *= np.float32(1e-44)
    x[1] *= np.float32(1e-40)
    x[2] *= np.float32(1e-38)
    x[3] *= np.float32(2e37)
    x[4, 3], x[5, 40], x[6, 127] = np.inf, -np.inf, np.nan
    x[7] = 0
    x[8] = -0.0
    x[9, :] = 0
    x[9, 64] = np.float32(1e-45)
    x[10, :32] = np.float32(3.0e38) * np.sign(x[10, :32])
    x[11] *= np.float32(1e-19)
    c, _ = make_cache(pk, rng, [0], 32, pk.PK_F32)
    t = torch.from_numpy(x).cuda()[None].contiguous()
    pk.pk_quant_append(c, t, t.flip(1).contiguous(), 12)
    kc, vc, ks, vs = ref.decode(c.tensors[0][0].cpu().numpy())
    k, v = torch.empty_like(t), torch.empty_like(t)
    pk.pk_quant_rows(c, 12, k, v)
    for code, s, y, back in ((kc, ks, x, k), (vc, vs, x[::-1], v)):
        want, scale, val = ref.stored(y)
        assert np.array_equal(s[:12], scale, equal_nan=True)
        live = np.repeat(scale > 0, 32, 1)
        assert np.array_equal(code[:12][live], want[live])
        with np.errstate(over="ignore", invalid="ignore"):
            assert np.array_equal(back[0].cpu().numpy(), val.astype(np.float32), equal_nan=True)


@gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("top", [1.0, 2.0 ** 126, 2.0 ** -56, 2.0 ** -57, 2.0 ** -58, 2.0 ** -126])
def test_append_every_bf16_value_of_a_group(pk, dtype, top):
    """Every bf16 value between a group's largest, of every mantissa, and its 64th part: all codes, borders and ties."""
    td, kind = dt(pk, dtype)
    big = np.float32(top) * (1 + np.arange(128, dtype=np.float32) / 128)
    steps = np.concatenate([np.float32(2.0 ** -e) * (1 + np.arange(128, dtype=np.float32) / 128) for e in range(7)])
    groups = []
    for m in big:
        x = np.float32(top) * steps
        x = np.sort(x[x <= m])[::-1] * np.where(np.arange((x <= m).sum()) % 2, -1, 1).astype(np.float32)
        x = np.concatenate([x, np.zeros(-len(x) % 31, np.float32)]).reshape(-1, 31)
        groups.append(np.concatenate([np.full((len(x), 1), m, np.float32), x], 1))
    g = np.concatenate(groups)
    g = np.concatenate([g, np.zeros((-len(g) % 4, 32), np.float32)])
    rows = torch.from_numpy(g.reshape(-1, D)).to(td)
    n = len(rows)
    cap = -(-n // KEYS) * KEYS
    c, _ = make_cache(pk, np.random.default_rng(0), [0], cap, kind)
    pk.pk_quant_append(c, rows.cuda()[None], rows.flip(0).contiguous().cuda()[None], n)
    kc, vc, ks, vs = ref.decode(c.tensors[0][0].cpu().numpy())
    for code, s, x in ((kc, ks, rows), (vc, vs, rows.flip(0))):
        want, scale, _ = ref.stored(x.float().numpy())
        assert np.array_equal(s[:n], scale)
        live = np.repeat(scale > 0, 32, 1)
        assert np.array_equal(code[:n][live], want[live])


@gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_append_at_places_and_refuses_what_does_not_fit(pk, dtype):
    td, kind = dt(pk, dtype)
    for n_new in (3, 70):                # one CTA per pair, several
        rng = np.random.default_rng(n_new)
        cap = 128
        lens = [50, 60, 70, 80, 90]
        c, before = make_cache(pk, rng, lens, cap, kind)
        at = torch.tensor([10, cap - n_new, cap - n_new + 1, -1, 0], dtype=torch.int32, device="cuda")
        x = make_rows(rng, 5 * n_new, td).view(5, n_new, D).cuda()
        pk.pk_quant_append(c, x, x, n_new, at=at)
        got = c.tensors[0].cpu().numpy()
        assert c.tensors[1].tolist() == [10 + n_new, cap, 70, 80, n_new]
        assert c.tensors[3][0].item() == pk._lib.PK_ERR_DEVICE_CHECK and c.tensors[3][1].item() in (2, 3)
        for p in (2, 3):
            assert np.array_equal(got[p], before[p])
        for p, a in ((0, 10), (1, cap - n_new), (4, 0)):
            k, v = ref.values(got[p])
            val = ref.stored(x[p].float().cpu().numpy())[2]
            assert np.array_equal(k[a:a + n_new], val) and np.array_equal(v[a:a + n_new], val)


@gpu
@pytest.mark.parametrize("n_new", [1, 40, 500])
@pytest.mark.parametrize("where", ["none", "lens"])
def test_append_places_that_are_the_lengths(pk, n_new, where):
    """at = None and at = lens itself append at the end; an `at` that overlaps lens in part is refused."""
    rng = np.random.default_rng(n_new)
    bh, cap = 3, 1024
    store = torch.tensor([7, 40, 100, 200], dtype=torch.int32, device="cuda")
    c, _ = make_cache(pk, rng, [0] * bh, cap, pk.PK_BF16)
    c = pk.pk_quant_view(c.tensors[0], store[:3], pk.PK_BF16)
    old = store[:3].tolist()
    x = make_rows(rng, bh * n_new, torch.bfloat16).view(bh, n_new, D).cuda()
    with pytest.raises(pk.PkError) as e:
        pk.pk_quant_append(c, x, x, n_new, at=store[1:])
    assert e.value.status == pk._lib.PK_ERR_INVALID_ARG
    pk.pk_quant_append(c, x, x, n_new, at=None if where == "none" else store[:3])
    got = c.tensors[0].cpu().numpy()
    assert store[:3].tolist() == [o + n_new for o in old]
    for p, o in enumerate(old):
        k, v = ref.values(got[p])
        val = ref.stored(x[p].float().cpu().numpy())[2]
        assert np.array_equal(k[o:o + n_new], val) and np.array_equal(v[o:o + n_new], val)


@gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("shift", [0, 1])
def test_rows_values_and_untouched_rows(pk, dtype, shift):
    td, kind = dt(pk, dtype)
    rng = np.random.default_rng(9)
    lens, n_rows = [0, 1, 33, 200], 100
    c, blocks = make_cache(pk, rng, lens, 224, kind)
    at = torch.tensor([0, 0, -5, 150], dtype=torch.int32, device="cuda")
    k = torch.full((4 * n_rows * D + shift,), 7.0, dtype=td, device="cuda")[shift:].view(4, n_rows, D)
    v = torch.full((4 * n_rows * D + shift,), 7.0, dtype=td, device="cuda")[shift:].view(4, n_rows, D)
    for a, use in ((at, at.tolist()), (None, [0] * 4)):
        k.fill_(7.0)
        v.fill_(7.0)
        pk.pk_quant_rows(c, n_rows, k, v, at=a)
        for p, n in enumerate(lens):
            kv = ref.values(blocks[p])
            for got, val in zip((k, v), kv):
                for i in range(n_rows):
                    slot = use[p] + i
                    want = torch.from_numpy(val[slot].astype(np.float32)).to(td) if 0 <= slot < n else torch.full((D,), 7.0, dtype=td)
                    assert torch.equal(got[p, i].cpu(), want), (p, i)


# ---------------------------------------------------------------- attention
def check_attend(pk, c, blocks, lens, q, G, scale=None, accumulate=False, acc0=None, calls=1):
    bh = len(lens)
    out = torch.full((bh, G, D), 5.0, device="cuda")
    lse = torch.full((bh, G), 5.0, device="cuda")
    work = torch.full((pk.pk_quant_attend_workspace(c, G, accumulate),), 0xff, dtype=torch.uint8, device="cuda")
    for _ in range(calls):
        pk.pk_quant_attend(c, q, G, out, work, lse=lse, accumulate=accumulate, scale=scale or 0.0)
    out, lse = out.cpu().double().numpy(), lse.cpu().double().numpy()
    for p, n in enumerate(lens):
        K, V = ref.values(blocks[p])
        o, l, w, eo, el, ew = ref.attend(q[p].double().cpu().numpy(), K[:n], V[:n], scale)
        assert np.all(np.abs(out[p] - o) <= eo), (p, n, np.max(np.abs(out[p] - o) / eo))
        if n:
            assert np.all(np.abs(lse[p] - l) <= el), (p, n, np.max(np.abs(lse[p] - l) / el))
        else:
            assert np.all(lse[p] == -np.inf)
        if accumulate:
            got = c.tensors[2][p].cpu().double().numpy()
            want = acc0[p].copy()
            want[:n] += calls * w.sum(0)
            # a rounding of the sum per call and head, and each weight's own error
            tol = calls * ((w * ew[:, None]).sum(0) + (G + 1) * ref.U * np.abs(want[:n])) + 1e-37
            assert np.all(np.abs(got[:n] - want[:n]) <= tol), (p, n, np.max(np.abs(got[:n] - want[:n]) / tol))
            assert np.array_equal(got[n:], acc0[p][n:])


@gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("G", [1, 2, 3, 4, 5, 8])
def test_attend_lengths_from_none_to_many(pk, dtype, G):
    td, kind = dt(pk, dtype)
    rng = np.random.default_rng(G)
    lens = [0, 1, 2, 31, 32, 33, 63, 64, 65, 0, 100, 1000, 1024, 0]
    acc0 = rng.random((len(lens), 1024)).astype(np.float32)
    c, blocks = make_cache(pk, rng, lens, 1024, kind, acc=acc0)
    q = make_rows(rng, len(lens) * G, td).view(len(lens), G, D).cuda()
    check_attend(pk, c, blocks, lens, q, G)
    check_attend(pk, c, blocks, lens, q, G, accumulate=True, acc0=acc0.astype(np.float64), calls=2)
    assert c.tensors[3].tolist() == [0, 0]


@gpu
@pytest.mark.parametrize("dtype,G,lens", [
    ("bf16", 4, [20011]), ("f32", 1, [4096]), ("f32", 8, [9001, 1, 0, 5000]), ("bf16", 8, [8192, 8191]),
    ("bf16", 1, [0]), ("f32", 3, [0, 0, 0]), ("bf16", 4, [577] * 300), ("f32", 2, [1] * 1500 + [40] * 3),
    ("f32", 5, [0, 700, 33] * 33), ("f32", 8, [90, 0, 31, 700] * 50), ("bf16", 7, [64] * 128), ("bf16", 6, [130] * 129),
    ("bf16", 3, [33] * 256), ("f32", 8, [65] * 257),
    ("bf16", 4, [(37 * i * i + 11 * i) % 3001 for i in range(100)]), ("f32", 7, [(53 * i * i + 7 * i) % 2500 for i in range(70)]),
    ("bf16", 5, [3000] * 60), ("f32", 2, [2100] * 100), ("f32", 7, [(37 * i * i + 11 * i) % 3001 for i in range(100)]),
    ("bf16", 2, [5000] * 100),
])
def test_attend_splits(pk, dtype, G, lens):
    """Long pairs over many workers, many pairs in one worker, nothing at all."""
    td, kind = dt(pk, dtype)
    rng = np.random.default_rng(len(lens) + G)
    cap = max(32, -(-max(lens) // KEYS) * KEYS)
    acc0 = np.zeros((len(lens), cap), np.float32)
    c, blocks = make_cache(pk, rng, lens, cap, kind, acc=acc0)
    q = (1.5 * make_rows(rng, len(lens) * G, td)).to(td).view(len(lens), G, D).cuda()
    check_attend(pk, c, blocks, lens, q, G, accumulate=True, acc0=acc0.astype(np.float64))
    check_attend(pk, c, blocks, lens, q, G, scale=0.011)


@gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_attend_q_off_the_boundary(pk, dtype):
    td, kind = dt(pk, dtype)
    rng = np.random.default_rng(12)
    c, blocks = make_cache(pk, rng, [70, 10], 96, kind)
    flat = torch.zeros(2 * 4 * D + 1, dtype=td, device="cuda")
    flat[1:] = make_rows(rng, 8, td).flatten().cuda()
    check_attend(pk, c, blocks, [70, 10], flat[1:].view(2, 4, D), 4)


@gpu
@pytest.mark.parametrize("G", [4, 6])
def test_attend_weights_off_the_boundary(pk, G):
    """acc that starts on a 4-byte boundary only."""
    rng = np.random.default_rng(14)
    lens = [70, 131, 3]
    c, blocks = make_cache(pk, rng, lens, 160, pk.PK_BF16)
    acc0 = rng.random((3, 160)).astype(np.float32)
    flat = torch.zeros(3 * 160 + 1, device="cuda")
    flat[1:] = torch.from_numpy(acc0).flatten().cuda()
    c = pk.pk_quant_view(c.tensors[0], c.tensors[1], pk.PK_BF16, acc=flat[1:].view(3, 160))
    q = make_rows(rng, 3 * G, torch.bfloat16).view(3, G, D).cuda()
    check_attend(pk, c, blocks, lens, q, G, accumulate=True, acc0=acc0.astype(np.float64))


@gpu
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("qs,vs", [(1e-3, 1.0), (40.0, 1.0), (1.0, 1e-25), (1.0, 1e25), (1e-30, 1e-10), (0.0, 1.0)])
def test_attend_magnitudes(pk, dtype, qs, vs):
    """Flat and one-hot softmax, tiny and huge values and queries."""
    td, kind = dt(pk, dtype)
    rng = np.random.default_rng(77)
    lens = [500, 33]
    acc0 = np.zeros((2, 512), np.float32)
    c, blocks = make_cache(pk, rng, lens, 512, kind, acc=acc0, v_scale=vs)
    q = (qs * make_rows(rng, 8, torch.float32)).to(td).view(2, 4, D).cuda()
    check_attend(pk, c, blocks, lens, q, 4, accumulate=True, acc0=acc0.astype(np.float64))


@gpu
def test_attend_values_of_mixed_size(pk):
    """Keys whose values are 2^40 or 2^-40 of their neighbours', zero rows, and a key of huge values that no query
    looks at: each contributes what its weight says."""
    rng = np.random.default_rng(8)
    n = 300
    K, V = make_rows(rng, n, torch.float32).numpy(), make_rows(rng, n, torch.float32).numpy()
    q = make_rows(rng, 4, torch.float32).numpy()
    V[::7] *= np.float32(2.0 ** -40)
    V[5] *= np.float32(2.0 ** 40)
    V[::11] = 0
    K[77] = -50 * q[0]                   # weight about e^-400 for head 0
    V[77] = 1e30
    K[78] = 0
    blocks = np.full((1, 10, BLOCK), 0xff, np.uint8)
    b = ref.pack(K, V)
    blocks[0, :len(b)] = b
    for kind, td in ((pk.PK_F32, torch.float32), (pk.PK_BF16, torch.bfloat16)):
        c = pk.pk_quant_view(torch.from_numpy(blocks).cuda(), torch.tensor([n], dtype=torch.int32, device="cuda"), kind)
        qq = torch.from_numpy(np.repeat(q[:1], 4, 0)).to(td).cuda()[None].contiguous()
        check_attend(pk, c, blocks, [n], qq, 4)


@gpu
def test_attend_long_tail_of_small_weights(pk):
    """One key 2^24 heavier than each of 300000 others whose values all point one way: the tail's share counts."""
    n, cap = 300001, 300032
    rng = np.random.default_rng(18)
    K, V = make_rows(rng, 64, torch.float32, 1e-3).numpy(), np.abs(make_rows(rng, 64, torch.float32).numpy())
    q = np.full((1, D), 0.5, np.float32)
    K[0] = 24 * math.log(2) * math.sqrt(D) / (0.5 * D)       # logit 24 ln 2; the others about 0
    K[32] = K[33]
    V[0] = 1
    two = ref.pack(K, V)
    blocks = np.concatenate([two[:1], np.repeat(two[1:], cap // KEYS - 1, 0)])[None]
    c = pk.pk_quant_view(torch.from_numpy(blocks).cuda(), torch.tensor([n], dtype=torch.int32, device="cuda"), pk.PK_F32)
    check_attend(pk, c, blocks, [n], torch.from_numpy(q)[None].cuda(), 1)


@gpu
def test_attend_nan_stays_in_its_group_of_values(pk):
    """A NaN group of V makes its 32 channels NaN and no others; a NaN group of K makes all of the pair NaN; rows
    behind the length (0xff bytes) and other pairs do not matter."""
    rng = np.random.default_rng(6)
    c, blocks = make_cache(pk, rng, [50, 50, 50], 64, pk.PK_F32, status=False)
    blocks[0, 0, 4352 + 8 * 9 + 2 * 1:][:2] = 0xff       # V scale of key 9, group 1
    blocks[1, 1, 4096 + 8 * 3 + 2 * 2:][:2] = 0xff       # K scale of key 35, group 2
    c.tensors[0].copy_(torch.from_numpy(blocks))
    q = make_rows(rng, 6, torch.float32).view(3, 2, D).cuda()
    out = torch.zeros(3, 2, D, device="cuda")
    pk.pk_quant_attend(c, q, 2, out, torch.empty(pk.pk_quant_attend_workspace(c, 2), dtype=torch.uint8, device="cuda"))
    out = out.cpu().double().numpy()
    K, V = ref.values(blocks[0])
    live = np.r_[0:32, 64:128]
    o, _, _, eo, _, _ = ref.attend(q[0].double().cpu().numpy(), K[:50], np.where(np.isnan(V[:50]), 0, V[:50]))
    assert np.isnan(out[0][:, 32:64]).all() and np.all(np.abs(out[0] - o)[:, live] <= eo[:, live])
    assert np.isnan(out[1]).all()
    K, V = ref.values(blocks[2])
    o, _, _, eo, _, _ = ref.attend(q[2].double().cpu().numpy(), K[:50], V[:50])
    assert np.all(np.abs(out[2] - o) <= eo)


@gpu
def test_attend_bad_lengths_are_clamped_and_recorded(pk):
    rng = np.random.default_rng(4)
    c, blocks = make_cache(pk, rng, [64, 64, 20], 64, pk.PK_BF16)
    c.tensors[1].copy_(torch.tensor([64, 65, -3], dtype=torch.int32))
    q = make_rows(rng, 3, torch.bfloat16).view(3, 1, D).cuda()
    check_attend(pk, c, blocks, [64, 64, 0], q, 1)
    assert c.tensors[3][0].item() == pk._lib.PK_ERR_DEVICE_CHECK and c.tensors[3][1].item() in (1, 2)


# ---------------------------------------------------------------- eviction
def check_evict(pk, src, blocks, lens, acc, dst_cap, kind, budget, sink, recent, with_acc=True, with_keep=True):
    bh = len(lens)
    fill = np.full((bh, dst_cap // KEYS, BLOCK), 0xA5, np.uint8)
    dst = pk.pk_quant_view(torch.from_numpy(fill).cuda(), torch.full((bh,), -9, dtype=torch.int32, device="cuda"), kind,
                           acc=torch.full((bh, dst_cap), 3.0, device="cuda") if with_acc else None)
    keep = torch.full((bh, budget), -7, dtype=torch.int32, device="cuda") if with_keep else None
    pk.pk_quant_evict(src, dst, budget, sink=sink, recent=recent, keep=keep)
    got = dst.tensors[0].cpu().numpy()
    assert np.array_equal(src.tensors[0].cpu().numpy(), blocks)
    for p, n in enumerate(lens):
        want = ref.evict(acc[p], n, budget, sink, recent)
        m = len(want)
        assert dst.tensors[1][p].item() == m
        if with_keep:
            assert np.array_equal(keep[p].cpu().numpy(), np.concatenate([want, np.full(budget - m, -1)]))
        if with_acc:
            assert np.array_equal(dst.tensors[2][p, :m].cpu().numpy(), acc[p][want], equal_nan=True)
            assert np.all(dst.tensors[2][p, m:].cpu().numpy() == 3.0)
        a, b, old = ref.decode(blocks[p]), ref.decode(got[p]), ref.decode(fill[p])
        for x, y, z in zip(a, b, old):
            assert np.array_equal(x[want], y[:m], equal_nan=True), (p, n)
            assert np.array_equal(y[m:], z[m:], equal_nan=True)


@gpu
@pytest.mark.parametrize("lens,budget,sink,recent", [
    ([0, 1, 2, 5], 1, 0, 0), ([0, 1, 2, 5], 1, 1, 0), ([7, 3, 64], 3, 1, 1), ([100, 90, 10], 40, 4, 36),
    ([100, 1000, 1023, 1024], 100, 3, 17), ([2000, 333, 999], 999, 64, 512), ([4096, 4095], 4094, 0, 0),
    ([5000] * 3, 32, 0, 32), ([3001, 20000], 1500, 64, 256),
])
@pytest.mark.parametrize("weights", ["heavy", "ties", "odd"])
def test_evict_keeps_the_heaviest(pk, lens, budget, sink, recent, weights):
    rng = np.random.default_rng(budget + len(lens))
    cap = -(-max(lens) // KEYS) * KEYS + 32
    bh = len(lens)
    if weights == "heavy":
        acc = np.exp(2 * rng.standard_normal((bh, cap)) - 5)
    elif weights == "ties":
        acc = rng.integers(0, 3, (bh, cap)) * 0.25
    else:                                # both zeros, negatives, infinities, NaN: an order all the same
        acc = rng.choice([0.0, -0.0, -1.0, np.inf, -np.inf, np.nan, 1e-45, -1e-45, 2.5], (bh, cap))
    acc = acc.astype(np.float32)
    src, blocks = make_cache(pk, rng, lens, cap, pk.PK_BF16, acc=acc)
    dst_cap = -(-min(budget, cap) // KEYS) * KEYS
    check_evict(pk, src, blocks, lens, acc, dst_cap, pk.PK_BF16, budget, sink, recent)
    check_evict(pk, src, blocks, lens, acc, dst_cap + 64, pk.PK_BF16, budget, sink, recent, with_acc=False, with_keep=False)


@gpu
def test_evict_long_rows(pk):
    """Longer than anything held on chip at once, the threshold's ties over the whole row."""
    rng = np.random.default_rng(3)
    n, cap = 300001, 300032
    blocks = torch.randint(0, 255, (2, cap // KEYS, BLOCK), dtype=torch.uint8, device="cuda")
    acc = np.exp(rng.standard_normal((2, cap))).astype(np.float32)
    acc[1] = rng.integers(0, 4, cap)
    src = pk.pk_quant_view(blocks, torch.tensor([n, n - 7], dtype=torch.int32, device="cuda"), pk.PK_F32,
                           acc=torch.from_numpy(acc).cuda())
    for budget in (1000, 200000):
        check_evict(pk, src, blocks.cpu().numpy(), [n, n - 7], acc, -(-budget // KEYS) * KEYS, pk.PK_F32, budget, 10, 300)


@gpu
@pytest.mark.parametrize("n,cap", [(16384, 16384), (16383, 16384), (16385, 16416), (40000, 40000), (131075, 131104)])
@pytest.mark.parametrize("shift", [0, 1])
def test_evict_sizes_at_the_borders(pk, n, cap, shift):
    """Around what a CTA holds at once; acc on 16-byte and on 4-byte boundaries; more pairs than CTAs fit."""
    bh = 300 if cap < 20000 else 3
    g = torch.Generator(device="cuda").manual_seed(n)
    flat = torch.randint(0, 1 << 14, (bh * cap + shift,), generator=g, device="cuda").float()
    acc = flat[shift:].view(bh, cap)
    blocks = torch.zeros(bh, cap // KEYS, BLOCK, dtype=torch.uint8, device="cuda")
    budget, sink, recent = 3000, 5, 100
    src = pk.pk_quant_view(blocks, torch.full((bh,), n, dtype=torch.int32, device="cuda"), pk.PK_BF16, acc=acc)
    dst = pk.pk_quant_view(torch.zeros(bh, 94, BLOCK, dtype=torch.uint8, device="cuda"), torch.zeros(bh, dtype=torch.int32, device="cuda"),
                           pk.PK_BF16, acc=torch.zeros(bh, 94 * KEYS, device="cuda"))
    keep = torch.zeros(bh, budget, dtype=torch.int32, device="cuda")
    pk.pk_quant_evict(src, dst, budget, sink=sink, recent=recent, keep=keep)
    mid = torch.sort(acc[:, sink:n - recent], dim=1, descending=True, stable=True).indices[:, :budget - sink - recent] + sink
    rest = torch.cat([torch.arange(sink, device="cuda"), torch.arange(n - recent, n, device="cuda")]).expand(bh, -1)
    want = torch.sort(torch.cat([mid, rest], 1), dim=1).values
    assert torch.equal(keep.long(), want) and torch.equal(dst.tensors[2][:, :budget], acc.gather(1, want))
    assert dst.tensors[1].tolist() == [budget] * bh


@gpu
@pytest.mark.parametrize("bh,n", [(20, 131104), (2, 270000), (20, 40000), (2, 131104), (1, 1048576), (1, 2100000), (17, 290001)])
@pytest.mark.parametrize("kind", ["equal", "few", "part", "near", "nan", "inf"])
def test_evict_crowded_weights(pk, bh, n, kind):
    """Weights that agree in their first bits: everywhere, in a part of the slots, or in all but the last bits."""
    budget, sink, recent = 2500, 7, 33
    cap = -(-n // KEYS) * KEYS
    g = torch.Generator(device="cuda").manual_seed(n)
    acc = torch.rand(bh, cap, generator=g, device="cuda")
    if kind == "equal":
        acc[:] = 0.25
    elif kind == "few":
        acc = torch.randint(0, 3, (bh, cap), generator=g, device="cuda").float()
    elif kind == "part":                 # the threshold falls on a value that fills one stretch
        acc *= 0.5
        acc[:, n // 3:n // 3 + 6000] = 0.75
        acc[:, 100:300] = 0.9
    elif kind == "near":
        acc = (0x3f800000 + torch.randint(0, 1 << 12, (bh, cap), generator=g, device="cuda", dtype=torch.int32)).view(torch.float32)
    elif kind == "nan":                  # the threshold is NaN: fewer others than the budget
        acc[:, 1000:] = float("nan")
    elif kind == "inf":
        acc[:, 500:9000] = float("inf")
    src = pk.pk_quant_view(torch.zeros(bh, cap // KEYS, BLOCK, dtype=torch.uint8, device="cuda"),
                           torch.full((bh,), n, dtype=torch.int32, device="cuda"), pk.PK_F32, acc=acc)
    dst = pk.pk_quant_view(torch.zeros(bh, 79, BLOCK, dtype=torch.uint8, device="cuda"), torch.zeros(bh, dtype=torch.int32, device="cuda"),
                           pk.PK_F32, acc=torch.zeros(bh, 79 * KEYS, device="cuda"))
    keep = torch.zeros(bh, budget, dtype=torch.int32, device="cuda")
    pk.pk_quant_evict(src, dst, budget, sink=sink, recent=recent, keep=keep)
    order = torch.where(acc.isnan(), float("-inf"), acc)[:, sink:n - recent]
    mid = torch.sort(order, dim=1, descending=True, stable=True).indices[:, :budget - sink - recent] + sink
    rest = torch.cat([torch.arange(sink, device="cuda"), torch.arange(n - recent, n, device="cuda")]).expand(bh, -1)
    want = torch.sort(torch.cat([mid, rest], 1), dim=1).values
    assert torch.equal(keep.long(), want)
    assert torch.equal(dst.tensors[2][:, :budget].view(torch.int32), acc.gather(1, want).view(torch.int32))


@gpu
@pytest.mark.parametrize("bh,n", [(3, 200), (3, 9000), (20, 40000), (2, 131104), (2, 2200000)])
@pytest.mark.parametrize("low,high,rest", [
    (0x3f800800, 0x3f800fff, 0x3f8007ff), (0x3f800800, 0x3f800fff, 0x3f000000), (0x00000000, 0x000007ff, 0x80000001),
    (0x00000800, 0x00000fff, 0x000007ff), (0x00000000, 0x00000000, 0x80000000), (0x80000000, 0x80000000, 0x80000800),
    (0xff800000, 0xff800000, 0x7fc00000), (0x7f800000, 0x7f800000, 0x7f7fffff), (0x007fffff, 0x00800000, 0x00000001),
])
def test_evict_threshold_at_the_border_of_a_digit(pk, bh, n, low, high, rest):
    """The kept weights are all those that share their first digits, or one less; the others lie right below."""
    count = 60
    cap = -(-n // KEYS) * KEYS
    g = torch.Generator(device="cuda").manual_seed(n)
    bits = torch.full((bh, cap), rest, dtype=torch.int64, device="cuda")
    for p in range(bh):
        at = torch.randperm(n, generator=g, device="cuda")[:count]
        bits[p, at] = torch.randint(low, high + 1, (count,), generator=g, device="cuda")
        bits[p, at[0]] = low
    acc = torch.where(bits > 0x7fffffff, bits - (1 << 32), bits).to(torch.int32).view(torch.float32)
    for budget in (count, count - 1, count + 1):
        src = pk.pk_quant_view(torch.zeros(bh, cap // KEYS, BLOCK, dtype=torch.uint8, device="cuda"),
                               torch.full((bh,), n, dtype=torch.int32, device="cuda"), pk.PK_F32, acc=acc)
        dst = pk.pk_quant_view(torch.zeros(bh, 2, BLOCK, dtype=torch.uint8, device="cuda"), torch.zeros(bh, dtype=torch.int32, device="cuda"), pk.PK_F32)
        keep = torch.zeros(bh, budget, dtype=torch.int32, device="cuda")
        pk.pk_quant_evict(src, dst, budget, keep=keep)
        for p in range(bh):
            assert keep[p].tolist() == ref.evict(acc[p, :n].cpu().numpy(), n, budget, 0, 0).tolist()


@gpu
@pytest.mark.parametrize("bh,n", [(1, 131104), (3, 1048576), (20, 40000), (40, 17000), (5, 9000)])
def test_evict_without_a_list(pk, bh, n):
    """Neither keep nor dst's acc: the same rows as with both, with keep alone and with acc alone."""
    cap = -(-n // KEYS) * KEYS
    g = torch.Generator(device="cuda").manual_seed(n)
    blocks = torch.randint(0, 256, (bh, cap // KEYS, BLOCK), generator=g, device="cuda", dtype=torch.uint8)
    src = pk.pk_quant_view(blocks, torch.full((bh,), n, dtype=torch.int32, device="cuda"), pk.PK_BF16,
                           acc=torch.randn(bh, cap, generator=g, device="cuda"))
    got = []
    for with_keep, with_acc in ((True, True), (False, False), (True, False), (False, True)):
        dst = pk.pk_quant_view(torch.zeros(bh, 63, BLOCK, dtype=torch.uint8, device="cuda"), torch.zeros(bh, dtype=torch.int32, device="cuda"),
                               pk.PK_BF16, acc=torch.zeros(bh, 63 * KEYS, device="cuda") if with_acc else None)
        keep = torch.zeros(bh, 2001, dtype=torch.int32, device="cuda") if with_keep else None
        pk.pk_quant_evict(src, dst, 2001, sink=9, recent=100, keep=keep)
        assert dst.tensors[1].tolist() == [2001] * bh
        got.append(dst.tensors[0])
    assert all(torch.equal(got[0], x) for x in got[1:])


# ---------------------------------------------------------------- together
@gpu
@pytest.mark.parametrize("G", [1, 5])
def test_rows_beyond_4_gigabytes(pk, G):
    """Pairs of 16 million keys, 7 GB: rows at their ends are written, attended, evicted and read back."""
    bh, n_cap, m = 3, (1 << 24) + 64, 40
    rng = np.random.default_rng(16)
    blocks = torch.zeros(bh, n_cap // KEYS, BLOCK, dtype=torch.uint8, device="cuda")      # scales of zero: keys and values of zero
    lens = torch.zeros(bh, dtype=torch.int32, device="cuda")
    c = pk.pk_quant_view(blocks, lens, pk.PK_F32, acc=torch.zeros(bh, n_cap, device="cuda"), status=torch.zeros(2, dtype=torch.int32, device="cuda"))
    K, V = make_rows(rng, bh * m, torch.float32).view(bh, m, D), make_rows(rng, bh * m, torch.float32).view(bh, m, D)
    at = torch.tensor([n_cap - m, n_cap - m - 7, n_cap - 2 * m], dtype=torch.int32, device="cuda")
    pk.pk_quant_append(c, K.cuda(), V.cuda(), m, at=at)
    n = [int(x) for x in lens.tolist()]
    assert n == [a + m for a in at.tolist()]
    Kq, Vq = (torch.from_numpy(np.stack([ref.stored(x[p].numpy())[2] for p in range(bh)])) for x in (K, V))
    k, v = torch.zeros(bh, m, D, device="cuda"), torch.zeros(bh, m, D, device="cuda")
    pk.pk_quant_rows(c, m, k, v, at=at)
    assert torch.equal(k.cpu().double(), Kq.float().double()) and torch.equal(v.cpu().double(), Vq.float().double())
    # logits of about 25 at the end against 16 million of zero
    q = torch.stack([K[:, (7 * g + 3) % m] for g in range(G)], 1)
    q = (q * (25 * math.sqrt(D) / (q * q).sum(-1, keepdim=True))).float()
    out, lse = torch.zeros(bh, G, D, device="cuda"), torch.zeros(bh, G, device="cuda")
    work = torch.empty(pk.pk_quant_attend_workspace(c, G, True), dtype=torch.uint8, device="cuda")
    pk.pk_quant_attend(c, q.cuda(), G, out, work, lse=lse, accumulate=True)
    acc = c.tensors[2]
    for p in range(bh):
        z = q[p].double() @ Kq[p].double().T / math.sqrt(D)
        total = torch.exp(z).sum(1) + (n[p] - m)
        w = torch.exp(z) / total[:, None]
        # fp32 logits up to 25 (1e-6 relative each: 3e-5 of a weight, 1e-5 of a product at most), sums of 2^24 terms
        assert torch.allclose(out[p].cpu().double(), w @ Vq[p].double(), rtol=0, atol=2e-4 * float(Vq.abs().max()))
        assert torch.allclose(lse[p].cpu().double(), torch.log(total), rtol=0, atol=2e-4)
        assert torch.allclose(acc[p, n[p] - m:n[p]].cpu().double(), w.sum(0), rtol=2e-4, atol=0)
        assert torch.allclose(acc[p, :n[p] - m].double().sum().cpu(), ((n[p] - m) / total).sum(), rtol=2e-4)
        assert acc[p, n[p]:].abs().max() == 0 if n[p] < n_cap else True
    e = pk.pk_quant_view(torch.zeros(bh, 2, BLOCK, dtype=torch.uint8, device="cuda"), torch.zeros(bh, dtype=torch.int32, device="cuda"), pk.PK_F32)
    keep = torch.zeros(bh, m, dtype=torch.int32, device="cuda")
    pk.pk_quant_evict(c, e, m, recent=m // 2, keep=keep)
    pk.pk_quant_rows(e, m, k, v)
    for p in range(bh):
        order = torch.sort(acc[p, :n[p] - m // 2], descending=True, stable=True).indices[:m - m // 2].sort().values
        want = torch.cat([order, torch.arange(n[p] - m // 2, n[p], device="cuda")])
        assert torch.equal(keep[p].long(), want)
        for i, slot in enumerate(want.tolist()):
            j = slot - (n[p] - m)
            assert torch.equal(k[p, i].cpu(), Kq[p, j].float() if j >= 0 else torch.zeros(D))
            assert torch.equal(v[p, i].cpu(), Vq[p, j].float() if j >= 0 else torch.zeros(D))
    assert c.tensors[3].tolist() == [0, 0]


@gpu
def test_first_calls_may_be_captured(pk):
    """A process whose first calls are recorded into a graph."""
    import subprocess
    import sys

    from tests.conftest import ROOT
    code = """
import torch, kv_cache_top_b200 as pk
bh, G = 2, 4
blocks = torch.zeros(bh, 4, 4608, dtype=torch.uint8, device='cuda')
c = pk.pk_quant_view(blocks, torch.zeros(bh, dtype=torch.int32, device='cuda'), pk.PK_F32, acc=torch.zeros(bh, 128, device='cuda'))
e = pk.pk_quant_view(torch.zeros_like(blocks), torch.zeros(bh, dtype=torch.int32, device='cuda'), pk.PK_F32, acc=torch.zeros(bh, 128, device='cuda'))
x = torch.randn(bh, 5, 128, device='cuda')
q, out = torch.randn(bh, G, 128, device='cuda'), torch.zeros(bh, G, 128, device='cuda')
k, v = torch.zeros(bh, 5, 128, device='cuda'), torch.zeros(bh, 5, 128, device='cuda')
work = torch.empty(pk.pk_quant_attend_workspace(c, G, True), dtype=torch.uint8, device='cuda')
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    pk.pk_quant_append(c, x, x, 5)
    pk.pk_quant_attend(c, q, G, out, work, accumulate=True)
    pk.pk_quant_evict(c, e, 4)
    pk.pk_quant_rows(e, 4, k, v)
g.replay(); g.replay()
torch.cuda.synchronize()
assert c.tensors[1].tolist() == [10, 10] and e.tensors[1].tolist() == [4, 4]
assert abs(float(c.tensors[2].sum()) - 2 * bh * G) < 1e-3 and torch.isfinite(out).all() and float(out.abs().sum()) > 0
print('captured')
"""
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert "captured" in r.stdout, r.stderr[-2000:]


@gpu
def test_calls_in_a_captured_graph_on_another_stream(pk):
    """append + attend + evict recorded once and replayed: the replay sees the lengths and rows of its time."""
    rng = np.random.default_rng(21)
    bh, G, cap = 3, 4, 128
    lens = [5, 0, 64]
    acc0 = np.zeros((bh, cap), np.float32)
    c, _ = make_cache(pk, rng, lens, cap, pk.PK_BF16, acc=acc0)
    e = pk.pk_quant_view(torch.zeros(bh, 1, BLOCK, dtype=torch.uint8, device="cuda"),
                         torch.zeros(bh, dtype=torch.int32, device="cuda"), pk.PK_BF16, acc=torch.zeros(bh, 32, device="cuda"))
    k, v = (torch.zeros(bh, 1, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    q = torch.zeros(bh, G, D, dtype=torch.bfloat16, device="cuda")
    out, lse = torch.zeros(bh, G, D, device="cuda"), torch.zeros(bh, G, device="cuda")
    work = torch.empty(pk.pk_quant_attend_workspace(c, G, True), dtype=torch.uint8, device="cuda")
    keep = torch.zeros(bh, 32, dtype=torch.int32, device="cuda")

    def step():
        pk.pk_quant_append(c, k, v, 1)
        pk.pk_quant_attend(c, q, G, out, work, lse=lse, accumulate=True)
        pk.pk_quant_evict(c, e, 32, sink=1, recent=4, keep=keep)

    start = [t.clone() for t in c.tensors[:3]]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()                           # warm up off the capture
        for t, s in zip(c.tensors, start):
            t.copy_(s)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    acc = acc0.astype(np.float64)
    for it in range(40):
        new = [make_rows(rng, bh, torch.bfloat16).view(bh, 1, D) for _ in range(2)]
        k.copy_(new[0])
        v.copy_(new[1])
        q.copy_(make_rows(rng, bh * G, torch.bfloat16).view(bh, G, D))
        graph.replay()
        blocks, o = c.tensors[0].cpu().numpy(), out.cpu().double().numpy()
        for p, n0 in enumerate(lens):
            n = n0 + it + 1
            assert c.tensors[1][p].item() == n
            K, V = ref.values(blocks[p])
            assert np.array_equal(K[n - 1], ref.stored(new[0][p].float().numpy())[2][0])
            assert np.array_equal(V[n - 1], ref.stored(new[1][p].float().numpy())[2][0])
            want, _, w, eo, _, _ = ref.attend(q[p].double().cpu().numpy(), K[:n], V[:n])
            assert np.all(np.abs(o[p] - want) <= eo)
            acc[p, :n] += w.sum(0)
            mine = c.tensors[2][p].cpu().numpy()
            assert np.allclose(mine[:n], acc[p, :n], rtol=1e-3, atol=1e-6)
            kept = ref.evict(mine, n, 32, 1, 4)
            assert np.array_equal(keep[p].cpu().numpy()[:len(kept)], kept) and e.tensors[1][p].item() == len(kept)
            ek, ev = ref.values(e.tensors[0][p].cpu().numpy())
            assert np.array_equal(ek[:len(kept)], K[kept]) and np.array_equal(ev[:len(kept)], V[kept])


@gpu
def test_two_streams_with_their_own_workspaces(pk):
    """Two calls at once over one cache that neither writes."""
    rng = np.random.default_rng(30)
    lens, G = [4000, 300, 17], 4
    c, blocks = make_cache(pk, rng, lens, 4000, pk.PK_F32)
    res, streams = [], [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for s in streams:
        q = make_rows(rng, 3 * G, torch.float32).view(3, G, D).cuda()
        out = torch.zeros(3, G, D, device="cuda")
        work = torch.empty(pk.pk_quant_attend_workspace(c, G), dtype=torch.uint8, device="cuda")
        torch.cuda.synchronize()
        res.append((q, out, work))
    for _ in range(5):
        for s, (q, out, work) in zip(streams, res):
            pk.pk_quant_attend(c, q, G, out, work, stream=s)
    torch.cuda.synchronize()
    for q, out, _ in res:
        for p, n in enumerate(lens):
            K, V = ref.values(blocks[p])
            o, _, _, eo, _, _ = ref.attend(q[p].double().cpu().numpy(), K[:n], V[:n])
            assert np.all(np.abs(out[p].cpu().double().numpy() - o) <= eo)


# ---------------------------------------------------------------- the bounded decode cache
def test_bounded_cache_refuses_bad_sizes(pk):
    from kv_cache_top_b200.bounded_cache import BoundedCache
    K = torch.zeros(1, 2, 5, D)
    for kw in (dict(budget=0), dict(budget=4, sink=3, recent=2), dict(budget=4, sink=-1, recent=0), dict(budget=4, sink=0, recent=0, update=0),
               dict(budget=4, sink=0, recent=0, group=9)):
        with pytest.raises(ValueError):
            BoundedCache(K, K, **{**dict(group=2), **kw})
    with pytest.raises(ValueError):
        BoundedCache(K.half(), K.half(), group=2, budget=4, sink=0, recent=0)
    with pytest.raises(ValueError):
        BoundedCache(K[0], K[0], group=2, budget=4, sink=0, recent=0)


@gpu
@pytest.mark.parametrize("dtype,T0,budget,sink,recent,update", [
    ("bf16", 40, 24, 2, 8, 16), ("f32", 300, 64, 4, 20, 33), ("bf16", 0, 8, 0, 0, 5), ("bf16", 33, 32, 32, 0, 1),
])
def test_bounded_cache_steps(pk, dtype, T0, budget, sink, recent, update):
    """A run of steps against a plain one: the stored values, the attention of every step, the accumulated weights and
    the tokens that each eviction keeps."""
    from kv_cache_top_b200.bounded_cache import BoundedCache
    td, _ = dt(pk, dtype)
    rng = np.random.default_rng(T0 + budget)
    B, H, G = 2, 2, 3
    bh = B * H
    rows = [make_rows(rng, bh * T0, td).view(B, H, T0, D) for _ in range(2)]
    c = BoundedCache(rows[0].cuda(), rows[1].cuda(), group=G, budget=budget, sink=sink, recent=recent, update=update)
    held = [[ref.stored(x.view(bh, T0, D)[p].float().numpy())[2] for x in rows] for p in range(bh)]
    pos = [np.arange(T0) for _ in range(bh)]
    acc = [np.zeros(T0) for _ in range(bh)]
    evictions = 0

    def check(q, out):
        out, lse = out.view(bh, G, D).cpu().double().numpy(), c.lse.view(bh, G).cpu().double().numpy()
        got = c.weights.reshape(bh, -1).cpu().double().numpy()
        for p in range(bh):
            o, l, w, eo, el, ew = ref.attend(q.view(bh, G, D)[p].double().numpy(), held[p][0], held[p][1])
            assert np.all(np.abs(out[p] - o) <= eo) and (not len(w[0]) or np.all(np.abs(lse[p] - l) <= el))
            acc[p] = acc[p] + w.sum(0)
            # every step's weights carry their bound and the sum a rounding: a relative part of what has been added
            tol = (ew.max(initial=0) * 2 + (G + 2) * ref.U * (c.T + 5)) * acc[p] + 1e-37
            assert np.all(np.abs(got[p] - acc[p]) <= tol)
            acc[p] = got[p].copy()                    # the next eviction goes by the kernel's sums

    for _ in range(3):
        q = make_rows(rng, bh * G, td).view(B, H * G, D)
        check(q, c.observe(q.cuda()))
    for t in range(3 * update + budget + 5):
        if c.n >= budget + update:
            evictions += 1
            for p in range(bh):
                keep = ref.evict(acc[p], c.n, budget, sink, recent)
                held[p] = [x[keep] for x in held[p]]
                pos[p], acc[p] = pos[p][keep], acc[p][keep]
        new = [make_rows(rng, bh, td).view(B, H, 1, D) for _ in range(2)]
        q = make_rows(rng, bh * G, td).view(B, H * G, D)
        out = c.step(q.cuda(), new[0].cuda(), new[1].cuda())
        for p in range(bh):
            held[p] = [np.concatenate([a, ref.stored(x.view(bh, 1, D)[p].float().numpy())[2]]) for a, x in zip(held[p], new)]
            pos[p], acc[p] = np.append(pos[p], T0 + t), np.append(acc[p], 0.0)
        check(q, out)
        assert c.evictions == evictions and c.T == T0 + t + 1
    assert evictions >= 3
    k, v = c.rows()
    where = c.positions.reshape(bh, -1).cpu().numpy()
    for p in range(bh):
        assert np.array_equal(where[p], pos[p])
        for got, want in ((k, held[p][0]), (v, held[p][1])):
            assert torch.equal(got.view(bh, -1, D)[p].cpu(), torch.from_numpy(want.astype(np.float32)).to(td))

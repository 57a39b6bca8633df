"""Appends to the FP8 and FP4 caches, byte for byte against quantisers that search
every code in exact arithmetic; untouched slots keep their bytes."""
import ctypes

import numpy as np
import pytest
import torch

import oracle
import paged_mqa_logits_b200 as mq
import workloads
from tests import cache_ref as ref

gpu = pytest.mark.gpu
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16}


def tokens(shape, dtype, seed):
    """Normal values of many sizes, with zero tokens, zero blocks, ties of both
    formats, the type's largest and its subnormal values among them."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(shape, generator=g) * torch.exp(2 * torch.randn(shape[:-1], generator=g))[..., None]
    flat = x.view(-1, shape[-1])
    n = flat.shape[0]
    ties = torch.tensor([6, .25, -.25, .75, 1.25, -1.75, 2.5, 3.5, -5, 5, .2, -.2, 0, -0., 1.5, 4])
    if n > 3:
        flat[0] = 0
        flat[1, :16] = 0
        flat[2] = ties.repeat(shape[-1] // 16)
        flat[3] = ties.repeat(shape[-1] // 16) * 7 / 64
    if n > 6:
        flat[4] = flat[4].sign() * torch.finfo(dtype).max
        flat[5] *= torch.finfo(dtype).tiny / 8
        flat[6] = torch.linspace(-1, 1, shape[-1]) * (3 / 1.75)
    return x.to(dtype)


def setup(ctx, ps, seed, width=None):
    """A shuffled block table with spare pages for rows of ctx tokens."""
    g = torch.Generator().manual_seed(seed)
    counts = [-(-max(c, 0) // ps) for c in ctx]
    P = sum(counts) + 2
    order = torch.randperm(P, generator=g).to(torch.int32)
    table = torch.full((len(ctx), width or max(max(counts), 1)), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(counts):
        table[b, :n] = order[at:at + n]
        at += n
    return table, P


def expected_fp4(cache, x, where, heads, ps):
    """The cache with tokens x [T, heads, D] written at where[t] = (page, slot) or None."""
    T, _, D = x.shape
    out = cache.copy()
    c = out.reshape(out.shape[0], heads, -1)
    codes, scales, vals = ref.quantise_fp4(x.double().numpy())
    for t, w in enumerate(where):
        if w is not None:
            p, s = w
            c[p, :, s * D // 2:(s + 1) * D // 2] = codes[t]
            at = ps * D // 2 + s * D // 16
            c[p, :, at:at + D // 16] = scales[t]
    return c.reshape(out.shape), vals


def expected_fp8(cache, x, where, ps):
    T, D = x.shape
    out = cache.copy()
    codes, s, vals = ref.quantise_fp8(x.double().numpy())
    for t, w in enumerate(where):
        if w is not None:
            p, slot = w
            out[p, slot * D:(slot + 1) * D] = codes[t]
            out[p, ps * D + 4 * slot:ps * D + 4 * slot + 4] = np.frombuffer(np.float32(s[t]).tobytes(), np.uint8)
    return out, vals


def places(table, ctx, offsets, T, ps, P, per_row=None):
    out = []
    for b, pos in ref.token_rows(ctx, offsets, T, per_row):
        ok = b >= 0 and 0 <= pos < table.shape[1] * ps
        page = int(table[b, pos // ps]) if ok else -1
        out.append((page, pos % ps) if 0 <= page < P else None)
    return out


CASES = [
    # new tokens a row, context after them, page size, D, heads, type
    ([1], [1], 16, 64, 1, "bf16"),
    ([1, 1, 1, 1], [1, 64, 65, 300], 64, 128, 1, "f16"),
    ([3, 0, 17, 1], [3, 40, 17, 129], 16, 128, 3, "bf16"),
    ([130, 1, 0, 0, 70], [200, 1, 0, 5, 256], 32, 64, 2, "f16"),
    ([257, 300], [257, 555], 256, 128, 1, "bf16"),
    ([9, 0], [9, 0], 128, 64, 8, "bf16"),
]


@gpu
@pytest.mark.parametrize("case", CASES, ids=[f"{len(c[0])}rows-p{c[2]}-d{c[3]}-h{c[4]}-{c[5]}" for c in CASES])
def test_fp4(case):
    new, ctx, ps, D, heads, dtype = case
    T = sum(new) + 3  # three tokens behind the last row
    table, P = setup(ctx, ps, seed=CASES.index(case))
    offsets = [0, *np.cumsum(new).tolist()]
    fused = tokens((T, 2, heads, D), TYPES[dtype], seed=5)
    g = torch.Generator().manual_seed(6)
    size = heads * ps * (D // 2 + D // 16)
    kc, vc = torch.randint(0, 256, (2, P, size), generator=g, dtype=torch.uint8)
    dev = fused.cuda()
    dk, dv = kc.cuda(), vc.cuda()
    kv = torch.full_like(dev[:, 0], 7.0).contiguous()
    vv = kv.clone()
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    mq.mqa_logits_clear_status()
    mq.mqa_cache_append_fp4(dev[:, 0], dev[:, 1], dk, dv, table.cuda(), i32(ctx), i32(offsets),
                            page_size=ps, k_values=kv, v_values=vv, flags=mq.MQA_FLAG_VALIDATE)
    where = places(table, ctx, offsets, T, ps, P)
    assert where[-3:] == [None] * 3
    for got, cache, x, vals in ((dk, kc, fused[:, 0], kv), (dv, vc, fused[:, 1], vv)):
        want, values = expected_fp4(cache.numpy(), x, where, heads, ps)
        np.testing.assert_array_equal(got.cpu().numpy(), want)
        for t in range(T):
            w = torch.from_numpy(values[t]).to(TYPES[dtype]) if where[t] else torch.full((heads, D), 7.0).to(TYPES[dtype])
            assert torch.equal(vals[t].cpu(), w)
    assert mq.mqa_logits_get_status() == 0


@gpu
@pytest.mark.parametrize("case", CASES, ids=[f"{len(c[0])}rows-p{c[2]}-d{c[3]}-{c[5]}" for c in CASES])
@pytest.mark.parametrize("small", [False, True])
def test_fp8(case, small):
    new, ctx, ps, D, _, dtype = case
    ps, D = (8, 32) if small else (ps, D)
    T = sum(new) + 2
    table, P = setup(ctx, ps, seed=CASES.index(case))
    offsets = [0, *np.cumsum(new).tolist()]
    x = tokens((T, D), TYPES[dtype], seed=8)
    g = torch.Generator().manual_seed(9)
    cache = torch.randint(0, 256, (P, ps * (D + 4)), generator=g, dtype=torch.uint8)
    dc = cache.cuda()
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    values = mq.mqa_cache_append_fp8(x.cuda(), dc, table.cuda(), i32(ctx), i32(offsets), page_size=ps,
                                     values=torch.full((T, D), 7.0, dtype=TYPES[dtype], device="cuda"))
    where = places(table, ctx, offsets, T, ps, P)
    want, vals = expected_fp8(cache.numpy(), x, where, ps)
    np.testing.assert_array_equal(dc.cpu().numpy(), want)
    for t in range(T):
        w = torch.from_numpy(vals[t]).to(TYPES[dtype]) if where[t] else torch.full((D,), 7.0).to(TYPES[dtype])
        assert torch.equal(values[t].cpu(), w), t


@gpu
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("first", [0, 1, 3])
def test_a_slice_of_the_offsets(fp8, first):
    """Some of a batch's rows, with their part of the offsets and the whole batch's tokens: those
    before the first row and behind the last have no row, and what is cached stays."""
    new, ctx, ps, D = [3, 5, 0, 2, 4], [40, 10, 7, 33, 4], 16, 64
    table, P = setup(ctx, ps, seed=3)
    offsets = [0, *np.cumsum(new).tolist()]
    off, table, ctx = offsets[first:5], table[first:4].contiguous(), ctx[first:4]
    T = offsets[-1]
    x = tokens((T, 1, D), torch.bfloat16, seed=12)
    g = torch.Generator().manual_seed(13)
    cache = torch.randint(0, 256, (P, ps * (D + 4) if fp8 else ps * 36), generator=g, dtype=torch.uint8)
    where = places(table, ctx, off, T, ps, P)
    assert where[:off[0]] == [None] * off[0] and where[-4:] == [None] * 4
    dc, values = cache.cuda(), torch.full((T, 1, D), 7.0, dtype=torch.bfloat16, device="cuda")
    args = [torch.as_tensor(a, dtype=torch.int32).cuda() for a in (table, ctx, off)]
    if fp8:
        mq.mqa_cache_append_fp8(x[:, 0].cuda(), dc, *args, page_size=ps, values=values[:, 0])
        want, vals = expected_fp8(cache.numpy(), x[:, 0], where, ps)
    else:
        mq.mqa_cache_append_fp4(x.cuda(), None, dc, None, *args, page_size=ps, k_values=values)
        want, vals = expected_fp4(cache.numpy(), x, where, 1, ps)
    np.testing.assert_array_equal(dc.cpu().numpy(), want)
    for t in range(T):
        w = torch.from_numpy(vals[t]).to(torch.bfloat16).view(D) if where[t] else torch.full((D,), 7.0).to(torch.bfloat16)
        assert torch.equal(values[t, 0].cpu(), w), t


@gpu
def test_even_rows_strides_and_keys_alone():
    """No offsets: T / B tokens a row; a strided slice of a projection; an FP4 cache
    of keys without values."""
    ctx, ps, D = [5, 2, 40], 16, 64
    table, P = setup(ctx, ps, seed=1)
    x = tokens((6, 3, 4, D), torch.bfloat16, seed=2)
    cache = torch.zeros(P, 2 * ps * 36, dtype=torch.uint8)
    dc = cache.cuda()
    dx = x.cuda()[:, 1, 1:3]
    assert mq.mqa_cache_append_fp4(dx, None, dc, None, table.cuda(),
                                   torch.tensor(ctx, dtype=torch.int32, device="cuda"), page_size=ps) is None
    where = places(table, ctx, None, 6, ps, P, per_row=2)
    want, _ = expected_fp4(cache.numpy(), x[:, 1, 1:3], where, 2, ps)
    np.testing.assert_array_equal(dc.cpu().numpy(), want)


@gpu
@pytest.mark.parametrize("D,dtype", [(32, "bf16"), (64, "f16"), (128, "bf16")])
def test_even_rows_fp8(D, dtype):
    """No offsets, a strided slice; rows whose first new tokens have no place."""
    ctx, ps = [5, 3, 40, 0, 1], 8
    table, P = setup(ctx, ps, seed=1)
    x = tokens((15, 2, D), TYPES[dtype], seed=2)
    cache = torch.randint(0, 256, (P, ps * (D + 4)), generator=torch.Generator().manual_seed(3), dtype=torch.uint8)
    dc = cache.cuda()
    assert mq.mqa_cache_append_fp8(x.cuda()[:, 1], dc, table.cuda(), torch.tensor(ctx, dtype=torch.int32, device="cuda")) is None
    where = places(table, ctx, None, 15, ps, P, per_row=3)
    assert where.count(None) == 3 + 2
    np.testing.assert_array_equal(dc.cpu().numpy(), expected_fp8(cache.numpy(), x[:, 1], where, ps)[0])


@gpu
@pytest.mark.parametrize("fp8", [False, True])
def test_tokens_without_a_place_are_not_written(fp8):
    """Positions before the row's start and behind its table, bad pages, lengths of 0:
    skipped in every mode, named in validate mode; the others are written."""
    ps, D = 16, 64
    ctx, offsets = [2, 40, 20, 0], [0, 4, 8, 12, 13]
    table = torch.tensor([[0, -1], [1, 2], [3, 99], [5, 6]], dtype=torch.int32)  # row 1: 40 > 32 tokens
    P, T = 7, 13
    x = tokens((T, 1, D), torch.bfloat16, seed=3)
    cache = torch.zeros(P, ps * (D + 4) if fp8 else ps * 36, dtype=torch.uint8)
    where = places(table, ctx, offsets, T, ps, P)
    assert where.count(None) == 2 + 4 + 4 + 1
    want = expected_fp8(cache.numpy(), x[:, 0], where, ps)[0] if fp8 else expected_fp4(cache.numpy(), x, where, 1, ps)[0]
    args = (table.cuda(), torch.tensor(ctx, dtype=torch.int32, device="cuda"), torch.tensor(offsets, dtype=torch.int32, device="cuda"))
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    for kw, bits in ((dict(), 0), (dict(flags=mq.MQA_FLAG_VALIDATE), mq.MQA_STATUS_BAD_PAGE | mq.MQA_STATUS_BAD_CONTEXT)):
        dc = cache.cuda()
        if fp8:
            mq.mqa_cache_append_fp8(x[:, 0].cuda(), dc, *args, page_size=ps, status=status, **kw)
        else:
            mq.mqa_cache_append_fp4(x.cuda(), None, dc, None, *args, page_size=ps, status=status, **kw)
        np.testing.assert_array_equal(dc.cpu().numpy(), want)
        assert int(status) == bits
    mq.mqa_logits_clear_status()


@gpu
def test_the_logits_read_what_was_appended():
    """Keys appended in two calls, then scored: the FP8 and FP4 logits against the oracle
    on the caches' bytes."""
    B, H, D, ps, L = 3, 64, 128, 64, 640
    lens = [600, 130, 77]
    for kind in ("fp8", "fp4"):
        wl = workloads.make_workload(kind, B, 1, H, D, ps, L, lens, seed=4)
        cache = torch.zeros_like(wl.kv_cache).cuda()
        x = torch.randn(sum(lens), D, generator=torch.Generator().manual_seed(5)).to(torch.bfloat16).cuda()
        rows = torch.split(x, lens)
        table = wl.block_table.cuda()
        first = [500, 64, 0]
        for a, b in ((torch.zeros(3, dtype=torch.int), torch.tensor(first)), (torch.tensor(first), torch.tensor(lens))):
            part = torch.cat([r[i:j] for r, i, j in zip(rows, a.tolist(), b.tolist())])
            off = torch.tensor([0, *(b - a).cumsum(0).tolist()], dtype=torch.int32, device="cuda")
            ctx = b.to(torch.int32).cuda()
            if kind == "fp8":
                mq.mqa_cache_append_fp8(part, cache, table, ctx, off)
            else:
                mq.mqa_cache_append_fp4(part[:, None], None, cache, None, table, ctx, off)
        wl.kv_cache = cache.cpu()
        from tests.helpers import compare, run
        out, _ = run(wl)
        want, absw = oracle.logits(wl)
        compare(out.cpu().numpy(), want, absw)
        assert int((wl.kv_cache != 0).sum()) > sum(lens) * D // 4


@gpu
def test_captured_with_a_padded_batch():
    """A graph with room for 64 tokens, replayed with fewer and more."""
    ps, D, B = 16, 128, 5
    x = torch.zeros(64, 1, D, dtype=torch.float16, device="cuda")
    ctx, off = (torch.zeros(n, dtype=torch.int32, device="cuda") for n in (B, B + 1))
    table = torch.arange(B * 8, dtype=torch.int32, device="cuda").view(B, 8).flip(1).contiguous()
    cache = torch.zeros(B * 8, ps * 72, dtype=torch.uint8, device="cuda")
    mq.mqa_cache_append_fp4(x, None, cache, None, table, ctx, off)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        mq.mqa_cache_append_fp4(x, None, cache, None, table, ctx, off)
    have = np.zeros(B, np.int64)
    want = cache.cpu().numpy()
    for step, new in enumerate(([1, 0, 30, 2, 9], [0, 64, 0, 0, 0], [1, 1, 1, 1, 1])):
        have += new
        fresh = tokens((64, 1, D), torch.float16, seed=20 + step)
        x.copy_(fresh)
        ctx.copy_(torch.from_numpy(have.astype(np.int32)))
        off.copy_(torch.tensor([0, *np.cumsum(new)], dtype=torch.int32))
        g.replay()
        where = places(table.cpu(), have.tolist(), off.tolist(), 64, ps, B * 8)
        want, _ = expected_fp4(want, fresh, where, 1, ps)
        np.testing.assert_array_equal(cache.cpu().numpy(), want)


# ---------------------------------------------------------------- refusals (CPU)
def params(**kw):
    base = dict(batch=2, num_tokens=4, num_kv_heads=1, head_dim=128, page_size=64, num_pages=4,
                max_pages_per_row=2, dtype=0, flags=0, reserved=0, k_stride_t=128, k_stride_h=128,
                v_stride_t=128, v_stride_h=128, status=None)
    base.update(kw)
    return mq.AppendParams(**base)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("kw,code,needle", [
    (dict(batch=-1), -1, "batch"), (dict(num_tokens=-1), -1, "num_tokens"),
    (dict(num_kv_heads=0), -1, "num_kv_heads"), (dict(head_dim=48), -4, "head_dim"),
    (dict(page_size=4), -1, "page_size"), (dict(page_size=24), -1, "page_size"),
    (dict(num_pages=0), -1, "num_pages"), (dict(max_pages_per_row=0), -1, "max_pages"),
    (dict(num_pages=2 ** 28), -4, "2^31"), (dict(dtype=5), -1, "dtype"),
    (dict(flags=0x100), -1, "flag"), (dict(k_stride_t=12), -1, "strides"),
    (dict(status=2), -1, "aligned"), (dict(num_tokens=2 ** 30), -4, "num_tokens"),
])
def test_bad_params(fp8, kw, code, needle):
    lib, p = mq.library(), params(**kw)
    if fp8:
        rc = lib.mqa_cache_append_fp8(16, 16, 16, 16, 16, None, ctypes.byref(p), None)
    else:
        rc = lib.mqa_cache_append_fp4(16, None, 16, None, 16, 16, 16, None, None, ctypes.byref(p), None)
    assert rc == code and needle in lib.mqa_logits_last_error().decode()


def test_bad_pointers_and_pairs():
    lib, p = mq.library(), params()

    def fp4(k=16, v=32, kc=48, vc=64, bt=16, ctx=16, off=16, kv=None, vv=None, p=p):
        return lib.mqa_cache_append_fp4(k, v, kc, vc, bt, ctx, off, kv, vv, ctypes.byref(p), None)

    def error():
        return lib.mqa_logits_last_error().decode()

    for name in ("k", "kc", "bt", "ctx"):
        assert fp4(**{name: None}) == -1 and "NULL" in error()
    for name in ("k", "v", "kc", "vc", "kv", "vv"):
        assert fp4(**{name: 24}) == -1 and "aligned" in error()
    for name in ("bt", "ctx", "off"):
        assert fp4(**{name: 18}) == -1 and "aligned" in error()
    assert fp4(v=None) == -1 and "together" in error()
    assert fp4(vc=48) == -1 and "two buffers" in error()
    assert fp4(v=None, vc=None, vv=16) == -1 and "v_values" in error()
    assert fp4(off=None, p=params(num_tokens=5)) == -1 and "multiple of batch" in error()
    assert fp4(p=params(num_tokens=0)) == 0 and fp4(p=params(batch=0)) == 0
    assert lib.mqa_cache_append_fp8(16, 16, 16, 16, 16, None, ctypes.byref(params(num_kv_heads=2)), None) == -1
    assert lib.mqa_cache_append_fp4(16, None, 16, None, 16, 16, 16, None, None, ctypes.byref(params(head_dim=32)), None) == -4
    assert lib.mqa_cache_append_fp8(16, 16, 16, 16, 16, None, None, None) == -1
    assert ctypes.sizeof(mq.AppendParams) == 80 and mq.AppendParams.k_stride_t.offset == 40


def test_overlapping_buffers():
    """Caches of 4 pages of 4608 bytes and values of 1024: overlapping by 16 bytes, refused."""
    lib, p = mq.library(), params()
    size = dict(kc=4 * 64 * 72, vc=4 * 64 * 72, kv=4 * 128 * 2, vv=4 * 128 * 2)
    good = dict(k=1 << 20, v=2 << 20, kc=3 << 20, vc=4 << 20, kv=5 << 20, vv=6 << 20)
    for x in size:
        for y in size:
            for at in () if x == y else (good[y], good[y] + size[y] - 16, good[y] - size[x] + 16):
                b = {**good, x: at}
                assert lib.mqa_cache_append_fp4(b["k"], b["v"], b["kc"], b["vc"], 16, 16, 16, b["kv"], b["vv"], ctypes.byref(p), None) == -1
                error = lib.mqa_logits_last_error().decode()
                assert "two buffers" in error if {x, y} == {"kc", "vc"} else "overlap" in error, (x, y, error)


def test_binding_checks_shapes():
    x = torch.zeros(4, 128, dtype=torch.bfloat16)
    k = x[:, None]
    c8, c4 = torch.zeros(4, 64 * 132, dtype=torch.uint8), torch.zeros(4, 64 * 72, dtype=torch.uint8)
    bt, ctx = torch.zeros(2, 2, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="x must"):
        mq.mqa_cache_append_fp8(k, c8, bt, ctx)
    with pytest.raises(ValueError, match="dtype"):
        mq.mqa_cache_append_fp8(x.float(), c8, bt, ctx)
    with pytest.raises(ValueError, match="pages hold"):
        mq.mqa_cache_append_fp8(x, c8, bt, ctx, page_size=32)
    with pytest.raises(ValueError, match="k must"):
        mq.mqa_cache_append_fp4(x, None, c4, None, bt, ctx)
    with pytest.raises(ValueError, match="together"):
        mq.mqa_cache_append_fp4(k, k, c4, None, bt, ctx)
    with pytest.raises(ValueError, match="shape and type"):
        mq.mqa_cache_append_fp4(k, k.half(), c4, c4, bt, ctx)
    with pytest.raises(ValueError, match="shape of k_cache"):
        mq.mqa_cache_append_fp4(k, k, c4, c4[:2], bt, ctx)
    with pytest.raises(ValueError, match="v_values"):
        mq.mqa_cache_append_fp4(k, None, c4, None, bt, ctx, v_values=k)
    with pytest.raises(ValueError, match="CUDA"):
        mq.mqa_cache_append_fp8(x, c8, bt, ctx)  # host tensors: no CPU path


def test_reference_quantisers():
    """The tests' own quantisers against torch's casts and the input recipe."""
    x = tokens((40, 64), torch.float16, seed=11).double()
    codes, s, vals = ref.quantise_fp8(x.numpy())
    t = (x / torch.from_numpy(s)[:, None]).float().to(torch.float8_e4m3fn)
    np.testing.assert_array_equal(t.view(torch.uint8).numpy(), codes)
    assert ((x.abs().amax(-1).numpy() / s <= 448) & ((x.abs().amax(-1).numpy() / s > 224) | (s == 1))).all()
    packed, sc, vals = ref.quantise_fp4(x.numpy())
    keep = x.abs().amax(-1) < 448 * 6  # the recipe of the inputs does not saturate its scales
    p2, s2 = workloads.encode_nvfp4(x[keep].float().unflatten(-1, (-1, 16)))
    np.testing.assert_array_equal(p2.numpy(), packed[keep.numpy()])
    np.testing.assert_array_equal(s2.numpy(), sc[keep.numpy()])

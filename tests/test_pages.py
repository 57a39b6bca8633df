"""Page operations against a plain model that takes one row after the other."""
import ctypes
import shutil
import threading

import numpy as np
import pytest
import torch

import paged_mqa_logits_b200 as mq
from tests import cache_ref as ref

gpu = pytest.mark.gpu


def pool(rng, B, W, ps, P, share=0.3, lens=None):
    """Tables of rows whose leading pages some rows share, and the pages' counts (with
    a few pages held by others than the tables)."""
    lens = rng.integers(0, W * ps + 1, B) if lens is None else np.array(lens)
    table = np.full((B, W), -1, np.int32)
    refs = np.zeros(P, np.int32)
    free = list(rng.permutation(P))
    for b in range(B):
        n = -(-int(lens[b]) // ps)
        twin = int(rng.integers(0, b)) if b and rng.random() < share else -1
        if twin >= 0:  # the twin's first tokens, the last page partly filled or not
            n_twin = -(-int(lens[twin]) // ps)
            lens[b] = min(lens[b], lens[twin]) if rng.random() < .7 else lens[b]
            n = -(-int(lens[b]) // ps)
        for j in range(n):
            if twin >= 0 and j < n_twin:
                table[b, j] = table[twin, j]
            elif free:
                table[b, j] = free.pop()
            else:
                lens[b], n = j * ps, j
                break
        for j in range(n):
            refs[table[b, j]] += 1
    for _ in range(min(2, len(free))):
        refs[free.pop()] = 1
    return table, lens.astype(np.int32), refs


def dev(*arrays):
    return [torch.from_numpy(np.array(a)).to(torch.int32).cuda() for a in arrays]


def same(got, want):
    for g, w in zip(got, want):
        np.testing.assert_array_equal(g.cpu().numpy(), w)


SHAPES = [(1, 1, 8, 2), (5, 4, 16, 30), (40, 9, 64, 500), (300, 3, 256, 1200), (7, 700, 8, 9000),
          (1500, 20, 32, 40001), (64, 1, 128, 64)]


@gpu
@pytest.mark.parametrize("B,W,ps,P", SHAPES)
@pytest.mark.parametrize("seed", [0, 1, 2])
def test_fork(B, W, ps, P, seed):
    rng = np.random.default_rng(seed)
    table, lens, refs = pool(rng, B, W, ps, P)
    R = [B, B + 3, max(1, B // 2)][seed]
    parents = rng.integers(-1, B, R).astype(np.int32)
    keep = rng.random(R) < .3
    parents[keep] = np.minimum(np.arange(R), B - 1)[keep]
    t, l, p, r = dev(table, lens, parents, refs)
    out = mq.mqa_pages_fork(t, l, p, r, page_size=ps)
    want = ref.fork(table, lens, parents, refs, ps)
    same((*out, r), want)
    same((t, l), (table, lens))


@gpu
@pytest.mark.parametrize("B,W,ps,P", SHAPES)
@pytest.mark.parametrize("seed", [0, 1, 2, 3])
def test_resize(B, W, ps, P, seed):
    """Growth, shrinking, both, and a pool that runs dry."""
    rng = np.random.default_rng(100 + seed)
    lens = rng.integers(0, W * ps + 1, B)
    if seed < 2:
        lens = lens // 2
    table, lens, refs = pool(rng, B, W, ps, P, share=.5, lens=lens)
    new = rng.integers(0, W * ps + 1, B)
    if seed == 0:
        new = np.minimum(lens + rng.integers(0, 5, B), W * ps)
    if seed == 3:  # few free pages: many rows are refused
        free = np.flatnonzero(refs == 0)
        refs[free[len(free) // 4:]] = 1
    t, l, n, r = dev(table, lens, new, refs)
    mq.mqa_logits_clear_status()
    src, dst = mq.mqa_pages_resize(t, l, n, r, page_size=ps)
    *want, ran_out = ref.resize(table, lens, new, refs, ps)
    same((t, l, r, src, dst), want)
    assert mq.mqa_logits_get_status() == (mq.MQA_STATUS_NO_PAGES if ran_out else 0)
    mq.mqa_logits_clear_status()


@gpu
@pytest.mark.parametrize("B,dry", [(24999, False), (25000, False), (25000, True), (32768, True)])
def test_resize_of_large_batches(B, dry):
    """Around the batch from which on a row's place is found again, with and without enough pages."""
    rng = np.random.default_rng(B + dry)
    ps, W = 16, 3
    table, lens, refs = pool(rng, B, W, ps, 3 * B)
    new = rng.integers(0, W * ps + 1, B)
    if dry:
        free = np.flatnonzero(refs == 0)
        refs[free[len(free) // 8:]] = 1
    t, l, n, r = dev(table, lens, new, refs)
    mq.mqa_logits_clear_status()
    src, dst = mq.mqa_pages_resize(t, l, n, r, page_size=ps)
    *want, ran_out = ref.resize(table, lens, new, refs, ps)
    same((t, l, r, src, dst), want)
    assert ran_out == dry and mq.mqa_logits_get_status() == (mq.MQA_STATUS_NO_PAGES if dry else 0)
    mq.mqa_logits_clear_status()


@gpu
def test_resize_with_the_pool_just_enough_and_one_short():
    ps = 16
    for spare in (0, 1):
        table = np.full((3, 4), -1, np.int32)
        table[0, 0], table[1, 0], table[2, 0] = 4, 4, 1
        refs = np.zeros(8 - spare, np.int32)
        refs[4], refs[1] = 2, 1
        lens, new = np.array([10, 10, 16]), np.array([40, 11, 33])  # need 3 (one in place of page 4), 1, 2
        t, l, n, r = dev(table, lens, new, refs)
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        src, dst = mq.mqa_pages_resize(t, l, n, r, page_size=ps, status=status)
        *want, ran_out = ref.resize(table, lens, new, refs, ps)
        assert ran_out == bool(spare) and int(status) == (mq.MQA_STATUS_NO_PAGES if spare else 0)
        same((t, l, r, src, dst), want)
        assert l.tolist() == ([40, 11, 33] if not spare else [40, 11, 16])
    mq.mqa_logits_clear_status()


@gpu
@pytest.mark.parametrize("B,W,ps,P", SHAPES)
@pytest.mark.parametrize("seed", [0, 1])
def test_compact(B, W, ps, P, seed):
    rng = np.random.default_rng(200 + seed)
    table, lens, refs = pool(rng, B, W, ps, P, lens=rng.integers(0, W * ps + 1, B) // (1 + seed))
    t, l, r = dev(table, lens, refs)
    src, dst, count, page_map = mq.mqa_pages_compact(t, l, r, page_size=ps)
    wt, wr, wsrc, wdst, wcount, wmap = ref.compact(table, lens, refs, ps)
    same((t, r, src, dst, page_map), (wt, wr, wsrc, wdst, wmap))
    assert count.tolist() == [wcount]


@gpu
@pytest.mark.parametrize("full", [0, 1])
def test_compact_of_an_empty_and_a_full_pool(full):
    for P in (1, 2, 3, 8193):
        t, l, r = dev(np.full((1, 1), -1), [0], np.full(P, full))
        src, dst, count, page_map = mq.mqa_pages_compact(t, l, r, page_size=8)
        assert count.tolist() == [0] and (src == -1).all() and (dst == -1).all()
        assert (r == full).all() and page_map.tolist() == (list(range(P)) if full else [-1] * P)


@gpu
@pytest.mark.parametrize("P,sizes", [(50, [16]), (300, [576, 4608, 33792]), (20, [4608 * 8 + 16]), (70, [48] * 9)])
def test_copy(P, sizes):
    g = torch.Generator().manual_seed(P)
    caches = [torch.randint(0, 256, (P, s), generator=g, dtype=torch.uint8) for s in sizes]
    order = torch.randperm(P, generator=g).to(torch.int32)
    n = P // 2
    src, dst = order[:n].clone(), order[n:2 * n].clone()
    holes = torch.rand(n, generator=g) < .2
    src[holes], dst[holes] = -1, -1
    for count in (None, 0, n // 2, n, n + 100):
        upto = n if count is None else min(count, n)
        want = [c.clone() for c in caches]
        for w, c in zip(want, caches):
            for s, d in zip(src[:upto].tolist(), dst[:upto].tolist()):
                if s >= 0:
                    w[d] = c[s]
        got = [c.cuda() for c in caches]
        mq.mqa_pages_copy(got if len(got) > 1 else got[0], src.cuda(), dst.cuda(),
                          None if count is None else torch.tensor([count], dtype=torch.int32, device="cuda"))
        for a, b in zip(got, want):
            assert torch.equal(a.cpu(), b)


@gpu
def test_bad_entries_are_skipped_and_reported():
    cache = torch.randint(0, 256, (4, 64), dtype=torch.uint8)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    for flags, bits in ((0, 0), (mq.MQA_FLAG_VALIDATE, mq.MQA_STATUS_BAD_PAGE)):
        got = cache.cuda()
        src, dst = dev([0, 9, 1, -3], [4, 1, 2, 0])
        mq.mqa_pages_copy(got, src, dst, flags=flags, status=status)
        want = cache.clone()
        want[2] = cache[1]
        assert torch.equal(got.cpu(), want) and int(status) == bits
        # tables with entries outside the pool, lengths outside the table, parents outside the batch
        status.zero_()
        table = np.array([[0, 77], [-5, 1], [2, 3]], np.int32)
        lens, refs = np.array([30, 32, 900]), np.array([1, 1, 1, 1, 0], np.int32)
        t, l, r, p = dev(table, lens, refs, [2, 0, 44, -7])
        out = mq.mqa_pages_fork(t, l, p, r, page_size=16, flags=flags, status=status)
        same((*out, r), ref.fork(table, lens, [2, 0, 44, -7], refs, 16))
        assert int(status) == (bits | mq.MQA_STATUS_BAD_CONTEXT if flags else 0)
        status.zero_()
        t, l, r, n = dev(table, lens, refs, [0, 33, 16])
        src, dst = mq.mqa_pages_resize(t, l, n, r, page_size=16, flags=flags, status=status)
        same((t, l, r, src, dst), ref.resize(table, lens, [0, 33, 16], refs, 16)[:5])
        assert int(status) == (bits | mq.MQA_STATUS_BAD_CONTEXT if flags else 0)
        status.zero_()
        t, l, r = dev(table, lens, refs)
        got = mq.mqa_pages_compact(t, l, r, page_size=16, flags=flags, status=status)
        wt, wr, wsrc, wdst, _, wmap = ref.compact(table, lens, refs, 16)
        same((t, r, got[0], got[1], got[3]), (wt, wr, wsrc, wdst, wmap))
        assert int(status) == (bits | mq.MQA_STATUS_BAD_CONTEXT if flags else 0)
        status.zero_()
    mq.mqa_logits_clear_status()


@gpu
def test_copies_of_no_page():
    """-1 on either side skips the pair without a word; other numbers outside the pool are named."""
    cache = torch.randint(0, 256, (4, 64), dtype=torch.uint8)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    for s, d, bits in ((-1, -1, 0), (-1, 2, 0), (2, -1, 0), (-1, 9, mq.MQA_STATUS_BAD_PAGE), (-2, 1, mq.MQA_STATUS_BAD_PAGE),
                       (4, -1, mq.MQA_STATUS_BAD_PAGE)):
        got = cache.cuda()
        mq.mqa_pages_copy(got, *dev([s], [d]), flags=mq.MQA_FLAG_VALIDATE, status=status.zero_())
        assert int(status) == bits and torch.equal(got.cpu(), cache), (s, d)
    mq.mqa_logits_clear_status()


@gpu
def test_unaligned_counts_and_a_captured_step():
    """page_refs as a view that starts off a 16-byte boundary; fork, resize, copy and
    compact captured once and replayed on other lengths."""
    rng = np.random.default_rng(5)
    B, W, ps, P = 30, 6, 16, 400
    cache = torch.randint(0, 256, (P, 4608), dtype=torch.uint8, device="cuda")
    buf = torch.zeros(P + 1, dtype=torch.int32, device="cuda")
    r = buf[1:]
    t, l, n, p = dev(np.full((B, W), -1), np.zeros(B), np.zeros(B), np.zeros(B))

    def step():
        t2, l2 = mq.mqa_pages_fork(t, l, p, r, page_size=ps)
        src, dst = mq.mqa_pages_resize(t2, l2, n, r, page_size=ps)
        mq.mqa_pages_copy(cache, src, dst)
        moves = mq.mqa_pages_compact(t2, l2, r, page_size=ps)
        mq.mqa_pages_copy(cache, *moves[:3])
        return t2, l2

    step()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = step()
    for _ in range(3):
        table, lens, refs = pool(rng, B, W, ps, P, share=.5, lens=rng.integers(0, W * ps - 8, B))
        parents = rng.integers(0, B, B).astype(np.int32)
        new = lens[parents] + rng.integers(0, 5, B)
        for d, a in zip((t, l, p, n, r), (table, lens, parents, new, refs)):
            d.copy_(torch.from_numpy(np.array(a)))
        cells = cache.clone().cpu().numpy()
        g.replay()
        ft, fl, fr = ref.fork(table, lens, parents, refs, ps)
        rt, rl, rr, src, dst, _ = ref.resize(ft, fl, new, fr, ps)
        for s, d in zip(src, dst):
            if s >= 0:
                cells[d] = cells[s]
        ct, cr, csrc, cdst, k, _ = ref.compact(rt, rl, rr, ps)
        cells[cdst[:k]] = cells[csrc[:k]]
        same((*out, r), (ct, rl, cr))
        np.testing.assert_array_equal(cache.cpu().numpy(), cells)


@gpu
def test_resize_of_large_batches_on_several_host_threads(tmp_path):
    """Batches whose shared memory is above the default, for the first time on every thread
    at once (a fresh copy of the library each round: what it has set up is its own)."""
    sizes, errors = (6000, 24000, 9000, 16000, 32768, 20000), []
    keep = [dev(*[np.zeros(B)] * 3, np.zeros(4), *[np.zeros(B)] * 2) for B in sizes]
    buffers = [[t.data_ptr() for t in tensors] for tensors in keep]
    for i in range(4):
        lib = ctypes.CDLL(shutil.copy(mq.library_path(), tmp_path / f"{i}.so"))
        lib.mqa_pages_resize.argtypes = mq.library().mqa_pages_resize.argtypes
        go = threading.Barrier(len(sizes))

        def work(B, at):
            p = params(batch=B, out_batch=0, max_pages_per_row=1, num_pages=4)
            go.wait()
            for _ in range(20):
                errors.append(lib.mqa_pages_resize(*at, ctypes.byref(p), None))

        threads = [threading.Thread(target=work, args=x) for x in zip(sizes, buffers)]
        for t in threads:
            t.start()
        for t in threads:
            t.join()
        torch.cuda.synchronize()
    assert len(errors) == 4 * 20 * len(sizes) and not any(errors)


@gpu
def test_streams_by_object_and_by_handle(monkeypatch):
    """The stream that the library is given: raw handles, 0 (the default stream) among
    them, streams, and the current one."""
    from paged_mqa_logits_b200 import cache as binding
    used, lib = [], mq.library()

    class Spy:
        @staticmethod
        def mqa_pages_copy(*args):
            used.append(args[-1])
            return lib.mqa_pages_copy(*args)

    monkeypatch.setattr(binding, "_library", Spy)
    pages = torch.zeros(4, 64, dtype=torch.uint8, device="cuda")
    src, dst = dev([0], [1])
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        for stream in (0, side.cuda_stream, torch.cuda.default_stream(), side, None):
            mq.mqa_pages_copy(pages, src, dst, stream=stream)
    assert used == [0, side.cuda_stream, 0, side.cuda_stream, side.cuda_stream]


# ---------------------------------------------------------------- refusals (CPU)
def params(**kw):
    base = dict(batch=2, out_batch=2, max_pages_per_row=4, num_pages=8, page_size=16, flags=0, status=None)
    base.update(kw)
    return mq.PagesParams(**base)


@pytest.mark.parametrize("kw,code,needle", [
    (dict(batch=-1), -1, "batch"), (dict(batch=40000), -1, "batch"), (dict(out_batch=-1), -1, "out_batch"),
    (dict(max_pages_per_row=0), -1, "max_pages"), (dict(num_pages=0), -1, "num_pages"),
    (dict(page_size=12), -1, "page_size"), (dict(page_size=4), -1, "page_size"), (dict(flags=64), -1, "flag"),
    (dict(status=6), -1, "aligned"), (dict(batch=30000, max_pages_per_row=100000), -4, "2^31"),
    (dict(num_pages=2 ** 30), -4, "2^31"),
])
def test_bad_params(kw, code, needle):
    lib, p = mq.library(), ctypes.byref(params(**kw))
    a = [1 << 20, 2 << 20, 3 << 20, 4 << 20, 5 << 20, 6 << 20, 7 << 20]
    for rc in (lib.mqa_pages_fork(*a[:6], p, None), lib.mqa_pages_resize(*a[:6], p, None),
               lib.mqa_pages_compact(*a, p, None)):
        assert rc == code
        assert needle in lib.mqa_logits_last_error().decode()


def test_bad_pointers():
    lib, p = mq.library(), ctypes.byref(params())
    a = [1 << 20, 2 << 20, 3 << 20, 4 << 20, 5 << 20, 6 << 20, 7 << 20]
    for fn, n in ((lib.mqa_pages_fork, 6), (lib.mqa_pages_resize, 6), (lib.mqa_pages_compact, 7)):
        for i in range(n):
            for bad, needle in ((None, "NULL"), (a[i] + 2, "aligned")):
                args = a[:n]
                args[i] = bad
                assert fn(*args, p, None) == -1 and needle in lib.mqa_logits_last_error().decode()
        assert fn(*a[:n], None, None) == -1
    assert lib.mqa_pages_fork(a[0], a[1], a[2], a[3], a[0] + 16, a[5], p, None) == -1
    assert "overlap" in lib.mqa_logits_last_error().decode()
    assert lib.mqa_pages_resize(a[0], a[1], a[1], a[3], a[4], a[5], p, None) == -1
    assert "overlap" in lib.mqa_logits_last_error().decode()
    assert lib.mqa_pages_resize(*[None] * 6, ctypes.byref(params(batch=0)), None) == 0
    assert lib.mqa_pages_fork(*[None] * 6, ctypes.byref(params(batch=0, out_batch=0)), None) == 0
    assert ctypes.sizeof(mq.PagesParams) == 32


def test_overlapping_buffers():
    """Every buffer that a call writes, against each of its others: overlapping by an entry, refused."""
    lib, p = mq.library(), params()  # tables of 32 bytes, lengths of 8, counts and maps of 32, lists of 16
    a = [i << 20 for i in range(1, 8)]
    size = dict(table=32, lens=8, refs=32, half=16, one=4)
    calls = ((lib.mqa_pages_fork, ("table", "lens", "lens", "refs", "table", "lens"), (3, 4, 5)),
             (lib.mqa_pages_resize, ("table", "lens", "lens", "refs", "lens", "lens"), (0, 1, 3, 4, 5)),
             (lib.mqa_pages_compact, ("table", "lens", "refs", "half", "half", "one", "refs"), (0, 2, 3, 4, 5, 6)))
    for fn, kinds, written in calls:
        for i in written:
            for j in range(len(kinds)):
                if i == j:
                    continue
                for at in (a[j], a[j] + size[kinds[j]] - 4, a[j] - size[kinds[i]] + 4):
                    args = a[:len(kinds)]
                    args[i] = at
                    assert fn(*args, ctypes.byref(p), None) == -1 and "overlap" in lib.mqa_logits_last_error().decode()


def test_copy_refusals():
    lib, p = mq.library(), ctypes.byref(params())

    def copy(ptrs=(16,), sizes=(64,), n=1, caches=None, src=16, dst=16, p=p, count=None):
        k = len(ptrs) if caches is None else caches
        return lib.mqa_pages_copy((ctypes.c_void_p * max(1, len(ptrs)))(*ptrs), (ctypes.c_int64 * max(1, len(sizes)))(*sizes),
                                  k, src, dst, n, count, p, None)

    for kw, needle in ((dict(n=-1), "n must"), (dict(caches=0), "num_caches"), (dict(caches=257), "num_caches"),
                       (dict(ptrs=(None,)), "aligned"), (dict(ptrs=(24,)), "aligned"), (dict(sizes=(0,)), "page_bytes"),
                       (dict(sizes=(72,)), "page_bytes"), (dict(src=None), "NULL"), (dict(dst=18), "aligned"),
                       (dict(count=18), "aligned"), (dict(p=ctypes.byref(params(num_pages=0))), "num_pages"),
                       (dict(p=None), "params")):
        assert copy(**kw) == -1 and needle in lib.mqa_logits_last_error().decode(), kw
    assert copy(n=0, src=None, dst=None) == 0


def test_binding_checks_shapes():
    t, l, r = torch.zeros(2, 4, dtype=torch.int32), torch.zeros(2, dtype=torch.int32), torch.zeros(8, dtype=torch.int32)
    c = torch.zeros(8, 64, dtype=torch.uint8)
    for call in (lambda: mq.mqa_pages_fork(t, l, l, r, page_size=16), lambda: mq.mqa_pages_resize(t, l, l, r, page_size=16),
                 lambda: mq.mqa_pages_compact(t, l, r, page_size=16), lambda: mq.mqa_pages_copy(c, l, l)):
        with pytest.raises(ValueError, match="CUDA"):
            call()
    with pytest.raises(ValueError, match="one shape"):
        mq.mqa_pages_copy(c, l, l[:1])
    with pytest.raises(ValueError, match="at least one"):
        mq.mqa_pages_copy([], l, l)

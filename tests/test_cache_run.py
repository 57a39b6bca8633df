"""The cache calls together, as a decode loop makes them: rows fork, grow, get pages
of their own, their new tokens go into an FP8 index cache and a 4-bit K and V, the
logits rank what each position sees, the attention reads the listed tokens, rows are
cut back, the pool is compacted. Checked after every step against the tokens that
each row should hold and the 64-bit references."""
import numpy as np
import pytest
import torch

import oracle
import paged_mqa_logits_b200 as mq
import workloads
from tests import cache_ref as ref
from tests.helpers import compare

gpu = pytest.mark.gpu
B, NEXT, INDEX_HEADS, HEADS, KV_HEADS, D, PS, P, W, K = 4, 2, 64, 12, 2, 128, 64, 40, 8, 96


class Loop:
    """The device's buffers, and one step of the loop on them."""

    def __init__(self):
        z = lambda *shape, dtype=torch.int32: torch.zeros(*shape, dtype=dtype, device="cuda")
        self.index = z(P, PS * (D + 4), dtype=torch.uint8)
        self.k, self.v = (z(P, KV_HEADS * PS * (D // 2 + D // 16), dtype=torch.uint8) for _ in range(2))
        self.table, self.lens, self.refs = torch.full_like(z(B, W), -1), z(B), z(P)
        # a step's inputs: each row's parent, length, new tokens (packed), queries
        self.parents, self.new, self.offsets = z(B), z(B), z(B + 1)
        self.xi = z(512, D, dtype=torch.bfloat16)
        self.xk, self.xv = (z(512, KV_HEADS, D, dtype=torch.bfloat16) for _ in range(2))
        self.qi = z(B, NEXT, INDEX_HEADS, D, dtype=torch.uint8)
        self.w = z(B, NEXT, INDEX_HEADS, dtype=torch.float32)
        self.q = z(B, NEXT, HEADS, D, dtype=torch.bfloat16)
        self.work = mq.mqa_attention_workspace(self.q, kv_heads=KV_HEADS)
        self.work_listed = mq.mqa_attention_workspace(self.q, kv_heads=KV_HEADS, topk=K)

    def caches(self):
        return self.index, self.k, self.v

    def state(self):
        return *self.caches(), self.table, self.lens, self.refs

    def grow(self):
        table, lens = mq.mqa_pages_fork(self.table, self.lens, self.parents, self.refs, page_size=PS)
        src, dst = mq.mqa_pages_resize(table, lens, self.new, self.refs, page_size=PS)
        mq.mqa_pages_copy(self.caches(), src, dst)
        self.table.copy_(table)
        self.lens.copy_(lens)
        mq.mqa_cache_append_fp8(self.xi, self.index, self.table, self.lens, self.offsets)
        mq.mqa_cache_append_fp4(self.xk, self.xv, self.k, self.v, self.table, self.lens, self.offsets)

    def answer(self):
        plan = mq.mqa_logits_schedule(self.lens)
        logits = mq.paged_mqa_logits_fp8(self.qi, self.index, self.table, self.lens, self.w, plan,
                                         page_size=PS, out_len=W * PS)
        picked = mq.mqa_logits_topk(logits, self.lens, K)
        args = dict(kv_heads=KV_HEADS, with_lse=True)
        listed = mq.paged_mqa_attention_fp4(self.q, self.k, self.v, self.table, self.lens, indices=picked,
                                            workspace=self.work_listed, **args)
        dense = mq.paged_mqa_attention_fp4(self.q, self.k, self.v, self.table, self.lens, plan,
                                           workspace=self.work, **args)
        return logits, picked, *listed, *dense

    def step(self):
        self.grow()
        return self.answer()

    def tidy(self, lens):
        """Rows cut back to `lens`, and the pool compacted."""
        src, dst = mq.mqa_pages_resize(self.table, self.lens, lens, self.refs, page_size=PS)
        assert (src == -1).all() and (dst == -1).all()
        moves = mq.mqa_pages_compact(self.table, self.lens, self.refs, page_size=PS)
        mq.mqa_pages_copy(self.caches(), *moves[:3])


class Rows:
    """What each row should hold: float64 [tokens, D] of the index, [tokens, KV_HEADS, D] of K and V."""

    def __init__(self):
        self.held = [(np.zeros((0, D)), np.zeros((0, KV_HEADS, D)), np.zeros((0, KV_HEADS, D))) for _ in range(B)]

    def step(self, loop, parents, new, rng):
        """Fills in a step's inputs and does the same to the rows."""
        self.held = [self.held[p] for p in parents]
        counts = [n - len(h[0]) for n, h in zip(new, self.held)]
        T = sum(counts)
        g = torch.Generator().manual_seed(int(rng.integers(1 << 30)))
        for x in (loop.xi, loop.xk, loop.xv):
            x.copy_(torch.randn(x.shape, generator=g) * 2)
        loop.qi.copy_((torch.randn(loop.qi.shape, generator=g)).to(torch.float8_e4m3fn).view(torch.uint8))
        loop.w.copy_(torch.randn(loop.w.shape, generator=g))
        loop.q.copy_(torch.randn(loop.q.shape, generator=g))
        off = [0, *np.cumsum(counts)]
        for d, a in ((loop.parents, parents), (loop.new, new), (loop.offsets, off)):
            d.copy_(torch.tensor(a, dtype=torch.int32))
        parts = (ref.quantise_fp8(loop.xi[:T].double().cpu().numpy())[2],
                 *(ref.quantise_fp4(x[:T].double().cpu().numpy())[2] for x in (loop.xk, loop.xv)))
        self.held = [tuple(np.concatenate((h, x[a:b])) for h, x in zip(held, parts))
                     for held, a, b in zip(self.held, off, off[1:])]

    def check(self, loop):
        """The caches hold the rows' tokens, and the counts are the tables' pointers."""
        index, k, v, table, lens, refs = (t.cpu().numpy() for t in loop.state())
        codes = index[:, :PS * D].reshape(P, PS, D)
        scale = index[:, PS * D:].copy().view(np.float32).astype(np.float64)
        value = np.where(codes >= 128, -1.0, 1.0) * ref.E4M3[codes & 127] * scale[..., None]
        kd, vd = (ref.decode_fp4(c, KV_HEADS, PS, D) for c in (k, v))
        assert lens.tolist() == [len(h[0]) for h in self.held]
        used = np.zeros(P, int)
        for b, (hi, hk, hv) in enumerate(self.held):
            t = np.arange(len(hi))
            page = table[b, t // PS]
            np.testing.assert_array_equal(value[page, t % PS], hi)
            np.testing.assert_array_equal(kd[page, :, t % PS], hk)
            np.testing.assert_array_equal(vd[page, :, t % PS], hv)
            np.add.at(used, table[b, :-(-len(hi) // PS)], 1)
        np.testing.assert_array_equal(refs, used)


def check_answer(loop, answer):
    logits, picked, listed, listed_lse, dense, dense_lse = answer
    k, v, table, lens, q = (t.cpu() for t in (loop.k, loop.v, loop.table, loop.lens, loop.q))
    wl = workloads.make_workload("fp8", B, NEXT, INDEX_HEADS, D, PS, W * PS, lens.tolist(), seed=0)
    wl.q, wl.kv_cache, wl.block_table, wl.context_lens, wl.weights = (
        t.cpu() for t in (loop.qi, loop.index, loop.table, loop.lens, loop.w))
    want, absw = oracle.logits(wl)
    compare(logits.cpu().numpy(), want, absw)
    sees = np.isfinite(want).sum(-1)
    x, at = logits.cpu().numpy(), picked.cpu().numpy()
    for b in range(B):
        for n in range(NEXT):
            m = min(K, int(sees[b, n]))
            order = np.lexsort((np.arange(W * PS), -x[b, n]))[:m]
            assert at[b, n].tolist() == order.tolist() + [-1] * (K - m)
    args = dict(heads_kv=KV_HEADS, ps=PS, scale=D ** -0.5)
    ref.check_attention(listed, listed_lse, ref.attention(q, k, v, table, lens, indices=picked.cpu(), **args),
                        K, torch.bfloat16)
    ref.check_attention(dense, dense_lse, ref.attention(q, k, v, table, lens, **args),
                        int(lens.max()), torch.bfloat16)


# parents and lengths of the loop's steps: prompts (one row empty), a beam step where
# one row's branches replace two others, decoding across a page's end, a row let go and
# a prompt in its place
STEPS = (([0, 1, 2, 3], [130, 64, 0, 200]),
         ([0, 0, 3, 3], [132, 131, 202, 202]),
         ([1, 0, 2, 3], [133, 134, 203, 263]))


@gpu
def test_a_decode_loop():
    mq.mqa_logits_clear_status()
    rng = np.random.default_rng(3)
    loop, rows = Loop(), Rows()
    for parents, new in STEPS:
        rows.step(loop, parents, new, rng)
        check_answer(loop, loop.step())
        rows.check(loop)
    cut = [133, 10, 0, 256]
    loop.tidy(torch.tensor(cut, dtype=torch.int32, device="cuda"))
    rows.held = [tuple(x[:n] for x in held) for held, n in zip(rows.held, cut)]
    rows.check(loop)
    live = int((loop.refs > 0).sum())
    assert not (loop.refs[live:] > 0).any()
    rows.step(loop, [0, 1, 2, 0], [135, 12, 300, 140], rng)
    check_answer(loop, loop.step())
    rows.check(loop)
    assert mq.mqa_logits_get_status() == 0


@gpu
def test_the_loop_captured_is_the_loop():
    """One step as a graph, on a stream of its own, replayed over the loop's inputs: every
    buffer and answer has the eager loop's bytes."""
    rng = np.random.default_rng(4)
    eager, graph, rows = Loop(), Loop(), Rows()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        graph.step()  # no rows yet: every context is empty
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        answer = graph.step()
    for parents, new in STEPS:
        rows.step(eager, parents, new, rng)
        for name in ("parents", "new", "offsets", "xi", "xk", "xv", "qi", "w", "q"):
            getattr(graph, name).copy_(getattr(eager, name))
        want = eager.step()
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            g.replay()
        side.synchronize()
        for a, b in zip((*graph.state(), *answer), (*eager.state(), *want)):
            assert torch.equal(a, b)
    rows.check(graph)

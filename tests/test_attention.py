"""Attention over the FP4 cache against a row-by-row reference in 64 bits, at the
lengths, masks, head layouts and lists where it can go wrong."""
import numpy as np
import pytest
import torch

import paged_mqa_logits_b200 as mq
from tests import cache_ref as ref

gpu = pytest.mark.gpu
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16}


class Case:
    """Inputs on the CPU: pages of a shuffled pool with spare pages; every slot that
    no row can see, and every spare page, holds NaN scales and full codes."""

    def __init__(self, ctx, nn, H, Hk, D, ps, dtype="bf16", seed=0, k=None, q_gain=2.0, spare=3,
                 width=None):
        g = torch.Generator().manual_seed(seed)
        self.ctx = torch.tensor(ctx, dtype=torch.int32)
        B = len(ctx)
        counts = [-(-max(c, 0) // ps) for c in ctx]
        width = width or max(max(counts), 1) + 1
        P = sum(counts) + spare
        order = torch.randperm(P, generator=g).to(torch.int32)
        self.table = torch.full((B, width), -1, dtype=torch.int32)
        at = 0
        for b, n in enumerate(counts):
            self.table[b, :n] = order[at:at + n]
            at += n
        self.nn, self.H, self.Hk, self.D, self.ps, self.dtype = nn, H, Hk, D, ps, TYPES[dtype]
        self.q = (q_gain * torch.randn(B, nn, H, D, generator=g)).to(self.dtype)
        self.k = self.pool(P, g)
        self.v = self.pool(P, g)
        seen = torch.zeros(P, ps, dtype=torch.bool)
        for b, c in enumerate(ctx):
            for t in range(max(c, 0)):
                seen[self.table[b, t // ps].long(), t % ps] = True
        for pool in (self.k, self.v):
            codes, scales = self.split(pool)
            codes[~seen[:, None].expand(-1, Hk, -1)] = 0xF7
            scales[~seen[:, None].expand(-1, Hk, -1)] = 0x7F
        self.indices = None
        if k:
            self.indices = torch.full((B, nn, k), -1, dtype=torch.int32)
            for b in range(B):
                for n in range(nn):
                    upto = min(max(ctx[b] - nn + 1 + n, 0), max(ctx[b], 0))
                    pick = torch.randperm(upto, generator=g)[:k] if upto else torch.zeros(0)
                    self.indices[b, n, :len(pick)] = pick.sort().values.to(torch.int32)
        self.scale = D ** -0.5

    def pool(self, P, g):
        x = torch.randn(P, self.Hk, self.ps, self.D, generator=g, dtype=torch.float64)
        x *= torch.exp(torch.randn(P, self.Hk, self.ps, 1, generator=g, dtype=torch.float64))
        codes, scales, _ = ref.quantise_fp4(x.numpy())
        both = np.concatenate((codes.reshape(P, self.Hk, -1), scales.reshape(P, self.Hk, -1)), -1)
        return torch.from_numpy(both.reshape(P, -1).copy())

    def split(self, pool):
        c = pool.view(pool.shape[0], self.Hk, -1)
        n = self.ps * self.D // 2
        return c[..., :n].unflatten(-1, (self.ps, self.D // 2)), c[..., n:].unflatten(-1, (self.ps, self.D // 16))

    def gpu(self):
        return {n: getattr(self, n).cuda() for n in ("q", "k", "v", "table", "ctx")} | \
            {"indices": None if self.indices is None else self.indices.cuda()}

    def call(self, d, num_ctas=None, **kw):
        sched = None if self.indices is not None else mq.mqa_logits_schedule(d["ctx"], num_ctas)
        return mq.paged_mqa_attention_fp4(d["q"], d["k"], d["v"], d["table"], d["ctx"], sched,
                                          kv_heads=self.Hk, scale=self.scale, indices=d["indices"],
                                          page_size=self.ps, **kw)

    def reference(self):
        return ref.attention(self.q, self.k, self.v, self.table, self.ctx, heads_kv=self.Hk,
                             ps=self.ps, scale=self.scale, indices=self.indices)

    def check(self, got, lse=None):
        T = max([1, *self.ctx.tolist()]) if self.indices is None else self.indices.shape[2]
        ref.check_attention(got, lse, self.reference(), T, self.dtype)

    def run_and_check(self, num_ctas=None):
        mq.mqa_logits_clear_status()
        out, lse = self.call(self.gpu(), num_ctas, with_lse=True)
        torch.cuda.synchronize()
        self.check(out, lse)
        assert mq.mqa_logits_get_status() == 0


DENSE = [
    # ctx, next_n, H, Hk, D, page size, type, CTAs
    ([1], 1, 1, 1, 64, 16, "bf16", None),
    ([0, 1, 2, 0, 3], 4, 2, 1, 128, 16, "f16", None),
    ([31, 32, 33, 63, 64, 65], 1, 8, 1, 128, 32, "bf16", None),
    ([255, 256, 257, 0, 511, 513], 2, 16, 2, 128, 64, "bf16", None),
    ([700, 5, 300], 3, 15, 3, 64, 16, "f16", 5),
    ([1000, 0, 129], 1, 32, 1, 128, 256, "f16", 2),
    ([640, 130, 1], 2, 64, 1, 128, 64, "bf16", 3),
    ([900], 1, 128, 1, 64, 128, "bf16", None),
    ([333, 90], 1, 34, 2, 64, 64, "bf16", 1),
    ([450, 17], 4, 24, 1, 128, 16, "bf16", None),
    ([777, 256], 1, 100, 1, 128, 64, "f16", 7),
    ([2500, 0, 0, 1200], 1, 7, 1, 128, 64, "bf16", 4),
    ([1600], 2, 8, 8, 64, 32, "f16", None),
    ([400] * 9, 1, 5, 5, 128, 16, "bf16", 148),
    ([600, 257], 1, 48, 1, 128, 16, "bf16", 3),
    ([1100, 3], 2, 33, 1, 64, 32, "f16", 4),
    ([520, 100, 256], 1, 65, 1, 64, 256, "bf16", 2),
    ([3000, 1], 4, 32, 1, 128, 64, "bf16", 6),
    # 17 to 128 rows a kv head, several heads and rows to a CTA, odd and even numbers of tiles
    ([333, 90, 128, 0, 1], 1, 51, 3, 128, 16, "f16", 1),
    ([128, 256, 129], 3, 44, 4, 64, 32, "bf16", 2),
    ([70, 513, 700], 2, 192, 3, 128, 64, "bf16", 4),
    ([1200, 5], 1, 80, 1, 128, 64, "f16", 3),
    ([300, 900, 77], 4, 40, 5, 64, 64, "bf16", 7),
]


@gpu
@pytest.mark.parametrize("case", DENSE, ids=[f"{c[0][0]}-n{c[1]}-h{c[2]}.{c[3]}-d{c[4]}-p{c[5]}" for c in DENSE])
def test_every_cached_token(case):
    *shape, dtype, ctas = case
    Case(*shape, dtype, seed=10 + DENSE.index(case)).run_and_check(ctas)


LISTS = [
    ([500, 0, 3, 70], 1, 8, 1, 128, 64, "bf16", 64),
    ([500, 1, 40], 3, 21, 3, 64, 16, "f16", 77),
    ([2000, 300], 2, 32, 1, 128, 64, "bf16", 1000),
    ([1500], 1, 128, 1, 128, 64, "f16", 513),
    ([64, 900], 4, 17, 1, 64, 32, "bf16", 31),
    ([40], 1, 1, 1, 64, 16, "bf16", 1),
    ([1200, 5], 1, 64, 1, 128, 64, "bf16", 300),
    ([800, 5], 1, 96, 2, 64, 256, "bf16", 200),
    ([700, 90, 0], 2, 60, 3, 128, 16, "f16", 300),
    ([400, 33], 1, 256, 2, 64, 64, "bf16", 129),
]


@gpu
@pytest.mark.parametrize("case", LISTS, ids=[f"{c[0][0]}-n{c[1]}-h{c[2]}.{c[3]}-d{c[4]}-k{c[7]}" for c in LISTS])
def test_listed_tokens(case):
    *shape, dtype, k = case
    Case(*shape, dtype, seed=40 + LISTS.index(case), k=k).run_and_check()


def many(B, most, seed):
    rng = np.random.default_rng(seed)
    return [int(c) for c in rng.integers(0, most + 1, B)]


MANY = [
    # more (head, part) pairs than CTAs, in batches whose rows give fewer parts than CTAs; more rows than CTAs
    (many(26, 7, 1), 2, 8, 8, 64, 16, "bf16", None, None),
    (many(3, 900, 2), 1, 64, 64, 64, 16, "f16", None, None),
    (many(20, 300, 3), 1, 144, 8, 128, 16, "bf16", None, None),
    (many(9, 600, 4), 4, 120, 5, 64, 32, "bf16", 16, None),
    (many(40, 30, 5), 1, 12, 12, 128, 64, "f16", 11, None),
    (many(300, 40, 6), 1, 6, 2, 128, 16, "bf16", None, None),
    (many(200, 300, 7), 1, 34, 2, 64, 16, "f16", None, None),
    # lists: more than SMs (one CTA each), and fewer, of lengths for one large CTA or several
    (many(40, 90, 8), 4, 12, 1, 128, 16, "bf16", None, 40),
    (many(160, 300, 9), 1, 5, 1, 64, 32, "f16", None, 210),
    (many(80, 300, 10), 2, 20, 2, 64, 16, "bf16", None, 130),
    (many(40, 500, 11), 1, 16, 2, 128, 16, "bf16", None, 300),
    (many(30, 900, 12), 1, 13, 1, 128, 64, "f16", None, 700),
    (many(30, 900, 13), 1, 3, 1, 64, 64, "bf16", None, 700),
    (many(20, 600, 14), 1, 10, 1, 64, 16, "f16", None, 500),
    # short lists of more than 16 query rows
    (many(50, 300, 15), 4, 75, 3, 64, 16, "bf16", None, 7),
    (many(3, 300, 16), 1, 112, 1, 128, 32, "f16", None, 100),
    (many(160, 300, 17), 1, 33, 1, 128, 16, "bf16", None, 128),
    (many(150, 200, 18), 1, 100, 1, 64, 64, "bf16", None, 60),
    # tables that hold one unit of the schedule a row
    (many(30, 112, 19), 2, 57, 3, 64, 16, "bf16", None, None),
    (many(170, 96, 20), 1, 33, 1, 128, 32, "f16", None, None),
    (many(9, 64, 21), 4, 4, 1, 128, 64, "bf16", 3, None),
    (many(12, 192, 22), 3, 62, 2, 64, 64, "f16", 30, None),
]


@gpu
@pytest.mark.parametrize("case", MANY, ids=[f"{len(c[0])}-n{c[1]}-h{c[2]}.{c[3]}-d{c[4]}-s{c[7]}-k{c[8]}" for c in MANY])
def test_many_rows_heads_and_lists(case):
    *shape, dtype, ctas, k = case
    Case(*shape, dtype, seed=70 + MANY.index(case), k=k).run_and_check(ctas)


@gpu
@pytest.mark.parametrize("nn,Hk,D,dtype", [(2, 1, 128, "bf16"), (3, 1, 64, "bf16"), (4, 2, 64, "f16")])
def test_lists_of_128_heads_and_several_positions(nn, Hk, D, dtype):
    """A list's tile holds one position's heads, whatever the number of positions."""
    Case([300, 1, 90, 0], nn, 128 * Hk, Hk, D, 64, dtype, seed=98 + nn, k=140).run_and_check()
    Case([1500], nn, 128 * Hk, Hk, D, 64, dtype, seed=98 + nn, k=1025).run_and_check()


@gpu
def test_lists_with_holes_repeats_and_tokens_out_of_sight():
    """-1 anywhere, tokens at and past the context, negatives, a token twice, and a
    position whose list is empty."""
    c = Case([300, 200, 90], 2, 8, 1, 128, 16, seed=60, k=100)
    g = torch.Generator().manual_seed(1)
    holes = torch.rand(c.indices.shape, generator=g) < 0.3
    c.indices[holes] = -1
    c.indices[0, 0, 3] = 299      # position 0 of two does not see the row's last token
    c.indices[0, 1, 3] = 300
    c.indices[0, 1, 4] = 2 ** 31 - 1
    c.indices[1, 0, 5:9] = -2 ** 31
    c.indices[1, 1, 10:14] = 17   # counted four times
    c.indices[2, 0] = -1
    c.run_and_check()
    c.indices[:, :, :] = -1
    d = c.gpu()
    out, lse = c.call(d, with_lse=True)
    assert not out.any() and torch.isneginf(lse).all()


@gpu
def test_scores_that_rise_along_the_row():
    """Every tile raises the running reference; large and tiny rows of q."""
    for rising in (1, -1):
        c = Case([1500, 700], 1, 20, 1, 128, 64, seed=61, q_gain=1.0)
        codes, scales = c.split(c.k)
        for b in range(2):
            t = torch.arange(int(c.ctx[b]))
            size = 60 + (t * 58 // int(c.ctx[b]) if rising > 0 else 58 - t * 58 // int(c.ctx[b]))
            scales[c.table[b][t // 64].long(), 0, t % 64] = size[:, None].to(torch.uint8)
        c.run_and_check()
    c = Case([300, 200, 100], 1, 4, 1, 128, 64, seed=62)
    q = c.q.float()
    q[0] *= 1e-20
    q[1] *= 2e4
    q[1, 0, 2] = 0
    c.q = q.to(torch.bfloat16)
    c.scale = 1e-5
    c.run_and_check()


LONG = [
    ([131072, 40001], 1, 8, 1, 128, 64, "bf16", None, None),
    ([100003], 1, 32, 2, 64, 256, "f16", 3, None),
    ([65537, 0, 5], 3, 10, 2, 128, 16, "bf16", 1, None),
    ([131072], 2, 64, 1, 128, 64, "bf16", 1, None),
    ([70000, 131071, 33], 4, 32, 1, 64, 16, "f16", None, None),
    ([50001], 1, 20, 1, 128, 128, "bf16", 7, None),
    ([131072, 9], 1, 8, 1, 128, 64, "f16", None, 60000),
    ([131072], 2, 40, 1, 64, 64, "bf16", None, 50001),
]


@gpu
@pytest.mark.parametrize("case", LONG, ids=[f"{c[0][0]}-n{c[1]}-h{c[2]}.{c[3]}-d{c[4]}-s{c[7]}-k{c[8]}" for c in LONG])
def test_long_rows(case):
    """Rows of tens of thousands of tokens, also in one CTA, with scores that rise along them."""
    ctx, nn, H, Hk, D, ps, dtype, ctas, k = case
    c = Case([1], nn, H, Hk, D, ps, dtype)
    g = torch.Generator(device="cuda").manual_seed(140 + LONG.index(case))
    B, P, W = len(ctx), sum(-(-n // ps) for n in ctx) + 2, -(-max(ctx) // ps)
    random = lambda lo, hi, *shape: torch.randint(lo, hi, shape, generator=g, device="cuda")  # noqa: E731
    order, at = torch.randperm(P, generator=g, device="cuda").to(torch.int32), 0
    d = {"table": torch.full((B, W), -1, dtype=torch.int32, device="cuda"),
         "ctx": torch.tensor(ctx, dtype=torch.int32, device="cuda"), "indices": None,
         "q": (2 * torch.randn(B, nn, H, D, generator=g, device="cuda")).to(c.dtype)}
    for n in "kv":
        d[n] = random(0, 256, P, Hk * ps * (D // 2 + D // 16)).to(torch.uint8)
        c.split(d[n])[1].copy_(random(0x28, 0x38, P, Hk, ps, D // 16))  # 0.25 to 0.9
    for b, n in enumerate(ctx):
        pages = order[at:at + -(-n // ps)]
        d["table"][b, :len(pages)] = pages
        at += len(pages)
        if n > 100:  # K grows along the row, to four times
            by = 16 * torch.arange(len(pages), device="cuda") // len(pages)
            c.split(d["k"])[1][pages.long()] += by[:, None, None, None].to(torch.uint8)
    if k:
        c.indices = d["indices"] = torch.stack([torch.stack([random(-2, max(n, 1), k) for _ in range(nn)]) for n in ctx]).to(torch.int32)
    out, lse = c.call(d, ctas, with_lse=True)
    table = torch.tensor([-1.0 if i >= 8 else 1.0 for i in range(16)], dtype=torch.float64, device="cuda") * \
        torch.tensor(list(ref.E2M1) * 2, dtype=torch.float64, device="cuda")
    scales = torch.tensor(ref.E4M3, dtype=torch.float64, device="cuda")
    want = [torch.zeros(B, nn, H, D, dtype=torch.float64, device="cuda"), torch.full((B, nn, H), -np.inf, dtype=torch.float64, device="cuda"),
            torch.zeros(B, nn, H, D, dtype=torch.float64, device="cuda"), torch.zeros(B, nn, H, dtype=torch.float64, device="cuda")]
    for b, n in enumerate(ctx):
        for i in range(nn):
            upto = max(n - nn + 1 + i, 0)
            t = torch.arange(upto, device="cuda")
            if k:
                t = d["indices"][b, i].long()
                t = t[(t >= 0) & (t < upto)]
            if not len(t):
                continue
            for h in range(Hk):
                kv = []
                for m in "kv":
                    codes, sc = (x[d["table"][b, t // ps].long(), h, t % ps] for x in c.split(d[m]))
                    both = torch.stack((codes & 15, codes >> 4), -1).flatten(1)
                    kv.append(table[both.long()] * scales[sc.long()].repeat_interleave(16, 1))
                qh = d["q"][b, i, h * (H // Hk):(h + 1) * (H // Hk)].double()
                x = c.scale * qh @ kv[0].T
                p, rows = torch.softmax(x, -1), (b, i, slice(h * (H // Hk), (h + 1) * (H // Hk)))
                want[0][rows], want[1][rows], want[2][rows] = p @ kv[1], torch.logsumexp(x, -1), p @ kv[1].abs()
                want[3][rows] = c.scale * (qh.abs() @ kv[0].abs().T).amax(-1) * 2.0 ** -16
    ref.check_attention(out, lse, [w.cpu().numpy() for w in want], max(ctx), c.dtype)


@gpu
@pytest.mark.parametrize("at", [0, 20000])
@pytest.mark.parametrize("heads", [8, 12, 32, 64, 128])
@pytest.mark.parametrize("listed", [False, True])
def test_a_sink_over_a_long_flat_row(listed, heads, at):
    """One token 17.5 nats above all others, whose v is 0: the result is what the others
    hold, 0.0034 (lists: 0.0009) of the mass, each p below 2^-25 of the largest. One CTA has
    the whole row."""
    T, D, ps, rows = (32768, 128, 64, 160) if listed else (131072, 128, 64, 1)
    c = Case([1], 1, heads, 1, D, ps)
    g = torch.Generator().manual_seed(96)
    q = 1 + torch.arange(heads) % 3 / 128
    c.q = q.to(torch.bfloat16)[None, None, :, None].expand(rows, 1, heads, D)
    c.scale = 17.5 / D
    c.k, c.v = (torch.zeros(T // ps, ps * (D // 2 + D // 16), dtype=torch.uint8) for _ in range(2))
    order = torch.randperm(T // ps, generator=g).to(torch.int32)
    c.table, c.ctx = order.expand(rows, -1).contiguous(), torch.full((rows,), T, dtype=torch.int32)
    page, slot = int(order[at // ps]), at % ps
    for pool in (c.k, c.v):
        codes, scales = c.split(pool)
        scales.fill_(0x38)  # 1
        if pool is c.v:
            codes.copy_(torch.randint(2, 5, codes.shape, generator=g) * 17)  # 1 to 2
        codes[page, 0, slot] = 0x22 if pool is c.k else 0  # every element 1 against 0; 0
    if listed:
        c.indices = torch.arange(T, dtype=torch.int32).expand(rows, 1, T).contiguous()
    got, lse = c.call(c.gpu(), 1, with_lse=True)
    assert torch.equal(got, got[:1].expand_as(got)) and torch.equal(lse, lse[:1].expand_as(lse))
    total = T - 1 + np.exp(17.5 * q.double().numpy())[:, None]
    o = ref.decode_fp4(c.v.numpy(), 1, ps, D).sum((0, 1, 2)) / total
    # the roundings of ref.check_attention, but an absolute one of p (three of them where P is
    # rescaled) is 2^-25 where the largest p is 2^7 at least, and moves o by |v - o| <= 2 of it
    err = 18 * 2.0 ** -16
    bound = 2.0 ** -8 * o + 2 * (err + 2.0 ** -11 + 2.0 ** -19) * o + T * 3 * 2.0 ** -32 * 2
    assert (np.abs(got[0, 0].double().cpu().numpy() - o) <= bound).all()
    assert (np.abs(lse[0, 0].double().cpu().numpy() - np.log(total[:, 0])) <= err + (T + 64) * 2.0 ** -24 + 2.0 ** -15).all()


@gpu
@pytest.mark.parametrize("heads", [6, 40])
@pytest.mark.parametrize("sign", [1, -1])
def test_scores_as_large_as_they_may_be(heads, sign):
    """Scores of up to 2^26, all of one sign or both: where one token stands out by more than the
    scores' error, its v is the result."""
    c = Case([1000, 40], 1, heads, 1, 128, 64, seed=97)
    codes, _ = c.split(c.k)
    if sign < 0:
        codes &= 0x77  # every k and q positive, the scale negative: every score is
        c.q = c.q.abs()
    c.scale = sign * 2.0 ** 22
    K = ref.decode_fp4(c.k.numpy(), 1, 64, 128)
    page = [c.table[b].numpy()[np.arange(n) // 64] for b, n in enumerate(c.ctx.tolist())]
    k = [K[p, 0, np.arange(len(p)) % 64] for p in page]
    top = max(np.abs(c.q[b, 0].double().numpy() @ x.T).max() for b, x in enumerate(k))
    c.q = (c.q * (15.9 / top)).to(torch.bfloat16)
    got, lse = c.call(c.gpu(), with_lse=True)
    assert torch.isfinite(got).all() and torch.isfinite(lse).all()
    V = ref.decode_fp4(c.v.numpy(), 1, 64, 128)
    clear = 0
    for b, p in enumerate(page):
        x = c.scale * c.q[b, 0].double().numpy() @ k[b].T
        assert np.abs(x).max() <= 2 ** 26
        order = np.argsort(-x, axis=1)
        err = abs(c.scale) * (np.abs(c.q[b, 0].double().numpy()) @ np.abs(k[b]).T).max(1) * 2.0 ** -16
        for h in range(heads):
            if x[h, order[h, 0]] - x[h, order[h, 1]] > 2 * err[h] + 100:
                t = order[h, 0]
                want = torch.from_numpy(V[p[t], 0, t % 64])
                assert torch.allclose(got[b, 0, h].double().cpu(), want, rtol=2 ** -8, atol=0), (b, h)
                assert abs(float(lse[b, 0, h]) - x[h, t]) <= err[h] + 2.0 ** -21 * abs(x[h, t])
                clear += 1
    assert clear >= heads


@gpu
@pytest.mark.parametrize("scale", [0.0, -0.125, 3.0])
def test_scales(scale):
    c = Case([290, 31], 2, 6, 2, 64, 32, "f16", seed=63, q_gain=0.5)
    c.scale = scale
    c.run_and_check()


NAN = [
    # the last tokens across the ends of spans, tiles, units of the schedule and pages
    ([257, 5, 1, 70], 2, 4, 1, 128, 16, "bf16", None),
    ([257, 514, 3], 3, 4, 2, 64, 32, "f16", 2),
    ([258, 33, 34], 4, 3, 1, 128, 16, "bf16", 148),
    ([64, 33, 34, 1, 2, 3], 2, 5, 5, 64, 32, "bf16", None),
    ([257, 100], 2, 16, 1, 128, 64, "bf16", None),
    ([257, 129, 2], 4, 16, 2, 128, 64, "f16", None),
    ([257, 600, 129, 3], 3, 20, 1, 64, 16, "bf16", 3),
    ([258, 514, 2], 4, 32, 1, 128, 64, "bf16", 2),
    ([130, 0, 257], 2, 40, 2, 64, 64, "f16", 1),
    # many rows to a CTA
    (many(40, 200, 31), 4, 24, 1, 128, 16, "bf16", 2),
    (many(40, 140, 32), 3, 60, 2, 64, 16, "f16", 1),
    (many(30, 300, 33), 2, 6, 1, 64, 16, "bf16", 1),
]


@gpu
@pytest.mark.parametrize("case", NAN, ids=[f"{c[0][0]}-n{c[1]}-h{c[2]}.{c[3]}-d{c[4]}-{c[6]}" for c in NAN])
def test_nan_that_later_positions_see(case):
    """NaN scales of V in a row's last tokens reach the blocks of 16 elements, and the
    positions, that see them, and no others."""
    *shape, dtype, ctas = case
    c = Case(*shape, dtype, seed=90 + NAN.index(case))
    clean, nn, D, ps = c.v.clone(), c.nn, c.D, c.ps
    nan = torch.zeros(len(c.ctx), nn, c.H, D, dtype=torch.bool)
    g = torch.Generator().manual_seed(3)
    codes, scales = c.split(c.v)
    _, safe = Case.split(c, clean)
    for b, ctx in enumerate(c.ctx.tolist()):
        for t in range(max(ctx - nn + 1, 0), ctx):
            page, s = int(c.table[b, t // ps]), t % ps
            for h in range(c.Hk):
                bad = torch.rand(D // 16, generator=g) < .4
                scales[page, h, s, bad] = 0x7F if t % 2 else 0xFF
                safe[page, h, s, bad] = 0
                for n in range(nn):
                    if t < ctx - nn + 1 + n:
                        nan[b, n, h * (c.H // c.Hk):(h + 1) * (c.H // c.Hk)] |= bad.repeat_interleave(16)
    assert nan.any() and not nan[:, 0].any()
    poisoned, c.v = c.v, clean
    want = c.reference()
    c.v = poisoned
    out, lse = c.call(c.gpu(), ctas, with_lse=True)
    assert torch.equal(out.isnan().cpu(), nan)
    got = torch.where(nan.cuda(), torch.from_numpy(want[0]).cuda().to(out.dtype), out)
    ref.check_attention(got, lse, want, int(c.ctx.max()), c.dtype)


@gpu
def test_strided_q_own_buffers_and_a_poisoned_workspace():
    c = Case([700, 0, 290], 2, 12, 2, 128, 64, seed=64)
    d = c.gpu()
    want, lse = c.call(d, with_lse=True)
    wide = torch.randn(3, 2, 3, 16, 128, device="cuda").to(torch.bfloat16)  # a fused projection's output
    view = wide[:, :, 1, 2:14]
    view.copy_(d["q"])
    assert not view.is_contiguous()
    work = mq.mqa_attention_workspace(view, kv_heads=2)
    work.view(torch.float32).fill_(float("nan"))
    out = torch.full_like(d["q"], float("nan"))
    d["q"] = view
    got, l2 = c.call(d, out=out, lse=torch.full_like(lse, float("nan")), workspace=work)
    assert got.data_ptr() == out.data_ptr()
    assert torch.equal(got, want) and torch.equal(l2, lse)
    c.check(got, l2)
    # one buffer for K and V
    c.v, d["v"] = c.k, d["k"]
    c.check(*c.call(d, with_lse=True))


@gpu
def test_bad_pages_are_clamped_and_reported():
    c = Case([300, 100], 1, 4, 1, 64, 16, seed=65, spare=0)
    c.table[0, 2] = c.k.shape[0] + 5
    c.table[1, 0] = -9
    d = c.gpu()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    for kw in ({}, {"flags": mq.MQA_FLAG_VALIDATE, "status": status}):
        out, lse = c.call(d, with_lse=True, **kw)
        c.check(out, lse)
    assert int(status) == mq.MQA_STATUS_BAD_PAGE
    mq.mqa_logits_clear_status()


@gpu
def test_lengths_beyond_the_table_and_negative_ones():
    c = Case([128, 64, 32], 1, 4, 1, 64, 16, seed=66, width=8)
    d = c.gpu()
    c.ctx[0], c.ctx[1] = 5000, -3   # the first row's table holds 128 tokens
    d["ctx"] = c.ctx.cuda()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    sched = mq.mqa_logits_schedule(d["ctx"])
    out, lse = mq.paged_mqa_attention_fp4(d["q"], d["k"], d["v"], d["table"], d["ctx"], sched,
                                          scale=c.scale, page_size=16, with_lse=True,
                                          flags=mq.MQA_FLAG_VALIDATE, status=status)
    assert int(status) & mq.MQA_STATUS_BAD_CONTEXT
    c.check(out, lse)
    mq.mqa_logits_clear_status()


@gpu
def test_stale_schedule_is_reported():
    c = Case([600, 300], 1, 4, 1, 64, 16, seed=67)
    d = c.gpu()
    sched = mq.mqa_logits_schedule(torch.tensor([600, 10], dtype=torch.int32, device="cuda"))
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    mq.paged_mqa_attention_fp4(d["q"], d["k"], d["v"], d["table"], d["ctx"], sched, page_size=16,
                               flags=mq.MQA_FLAG_VALIDATE, status=status)
    assert int(status) & mq.MQA_STATUS_STALE_SCHEDULE
    mq.mqa_logits_clear_status()


@gpu
@pytest.mark.parametrize("heads,ctas", [(8, None), (64, None), (1, 600), (5, 3)])
def test_validation_with_more_and_fewer_ctas_than_parts(heads, ctas):
    c = Case([600, 0, 300], 2, heads, heads, 64, 16, seed=68)
    d = c.gpu()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    for lens, stale in ((c.ctx, 0), (torch.tensor([600, 0, 10], dtype=torch.int32), mq.MQA_STATUS_STALE_SCHEDULE)):
        sched = mq.mqa_logits_schedule(lens.cuda(), ctas)
        out = mq.paged_mqa_attention_fp4(d["q"], d["k"], d["v"], d["table"], d["ctx"], sched, page_size=16,
                                         kv_heads=heads, scale=c.scale, flags=mq.MQA_FLAG_VALIDATE, status=status)
        assert int(status) == stale
        if not stale:
            c.check(out)
    mq.mqa_logits_clear_status()


@gpu
@pytest.mark.parametrize("k", [None, 600], ids=["all", "list"])
def test_captured_replayed_and_on_another_stream(k):
    """A replay follows new lengths, queries and cache contents; two graphs with a
    workspace each, and a call on a stream of its own, give the eager results."""
    a, b = (Case(x, 2, 16, 1, 128, 64, seed=70 + i, k=k, width=20)
            for i, x in enumerate(([900, 0, 300], [100, 1200, 513])))
    P = max(a.k.shape[0], b.k.shape[0])
    grow = lambda t: torch.cat((t, torch.full((P - t.shape[0], t.shape[1]), 0x7F, dtype=torch.uint8)))  # noqa: E731
    for c in (a, b):
        c.k, c.v = grow(c.k), grow(c.v)
    da, db = a.gpu(), b.gpu()
    want = [c.call(d, with_lse=True) for c, d in ((a, da), (b, db))]
    a.check(*want[0])
    b.check(*want[1])
    live = [{n: None if t is None else t.clone() for n, t in da.items()} for _ in range(2)]
    graphs, outs = [], []
    side = torch.cuda.Stream()
    for d in live:
        work = mq.mqa_attention_workspace(d["q"], topk=k or 0)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            outs.append(a.call(d, with_lse=True, workspace=work))
        graphs.append(g)
    for src, w in ((da, want[0]), (db, want[1]), (da, want[0])):
        for d in live:
            for n, t in d.items():
                if t is not None:
                    t.copy_(src[n])
        torch.cuda.synchronize()
        streams = [torch.cuda.Stream() for _ in graphs]
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for o in outs:
            assert torch.equal(o[0], w[0]) and torch.equal(o[1], w[1])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    sched = None if k else mq.mqa_logits_schedule(db["ctx"])
    s.wait_stream(torch.cuda.current_stream())
    got = mq.paged_mqa_attention_fp4(db["q"], db["k"], db["v"], db["table"], db["ctx"], sched,
                                     scale=b.scale, indices=db["indices"], page_size=64, stream=s)
    s.synchronize()
    assert torch.equal(got, want[1][0])


@gpu
def test_calls_on_several_streams_at_once():
    """Every kernel (wide, narrow, small CTAs, joined and not) on a stream and with a
    workspace of its own, all under way together: the bytes of the calls one by one."""
    shapes = [(([900, 30, 700], 2, 64, 1, 128, 64), None), (([500] * 9, 1, 48, 8, 64, 16), None),
              (([800, 300], 1, 12, 1, 128, 32), None), ((many(200, 200, 3), 1, 8, 1, 64, 16), 150),
              (([600] * 4, 1, 8, 1, 128, 64), 2048)]
    runs = []
    for i, (shape, k) in enumerate(shapes):
        c = Case(*shape, seed=120 + i, k=k)
        d = c.gpu()
        work = mq.mqa_attention_workspace(d["q"], kv_heads=c.Hk, topk=k or 0)
        runs.append((c, d, work, torch.cuda.Stream(), c.call(d, workspace=work, with_lse=True)))
    torch.cuda.synchronize()
    got = []
    for _ in range(10):
        for c, d, work, stream, _ in runs:
            with torch.cuda.stream(stream):
                got.append(c.call(d, workspace=work, with_lse=True))
    torch.cuda.synchronize()
    for i, (out, lse) in enumerate(got):
        want = runs[i % len(runs)][4]
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1])


@gpu
def test_pages_behind_four_gigabytes():
    """Byte offsets past 2^32 in a pool of 9 million pages."""
    c = Case([200, 90], 1, 8, 1, 64, 16, seed=80)
    P = 9_000_000
    assert P * c.k.shape[1] > 2 ** 32
    big = torch.empty(P, c.k.shape[1], dtype=torch.uint8, device="cuda")
    d = c.gpu()
    n = c.k.shape[0]
    big[P - n:] = d["k"]
    d["k"] = d["v"] = big
    c.v = c.k
    d["table"] = torch.where(d["table"] >= 0, d["table"] + (P - n), -1).to(torch.int32)
    out, lse = c.call(d, with_lse=True)
    c.check(out, lse)


@gpu
def test_position_of_the_split_changes_nothing_but_rounding():
    """Every number of CTAs covers every token once; the same call twice is the same."""
    c = Case([3000, 17, 1024], 2, 8, 1, 128, 64, seed=81)
    d = c.gpu()
    for ctas in (1, 2, 3, 13, 148, 300):
        out, lse = c.call(d, ctas, with_lse=True)
        again, l2 = c.call(d, ctas, with_lse=True)
        assert torch.equal(out, again) and torch.equal(lse, l2)
        c.check(out, lse)


@gpu
@pytest.mark.parametrize("k", [None, 129, 300, 777, 2048])
@pytest.mark.parametrize("heads,Hk,D", [(8, 1, 128), (21, 3, 64), (40, 1, 128)])
def test_a_workspace_serves_smaller_batches_and_fewer_positions(k, heads, Hk, D):
    """Its size never falls with the batch or the positions; one of a large batch serves a call of one row."""
    size = np.array([[mq.mqa_attention_workspace(torch.empty(B, n, heads, D, dtype=torch.float16, device="cuda"),
                                                 kv_heads=Hk, topk=k or 0).numel()
                      for B in (1, 2, 3, 5, 8, 13, 30, 70, 74, 75, 148, 149, 400)] for n in (1, 2, 3)])
    assert (np.diff(size, axis=0) >= 0).all() and (np.diff(size, axis=1) >= 0).all()
    c = Case([800], 2, heads, Hk, D, 64, seed=99, k=k)
    work = mq.mqa_attention_workspace(torch.empty(400, 3, heads, D, dtype=torch.float16, device="cuda"), kv_heads=Hk, topk=k or 0)
    c.check(c.call(c.gpu(), workspace=work))


# ---------------------------------------------------------------- refusals (CPU)
def params(**kw):
    base = dict(batch=2, next_n=1, num_heads=8, num_kv_heads=2, head_dim=128, page_size=64,
                num_pages=4, max_pages_per_row=2, topk=0, num_ctas=148, dtype=0, flags=0,
                softmax_scale=1.0, reserved=0, q_stride_b=1024, q_stride_n=1024, q_stride_h=128,
                workspace_bytes=1 << 40, status=None)
    base.update(kw)
    return mq.AttentionParams(**base)


@pytest.mark.parametrize("kw,code,needle", [
    (dict(batch=-1), -1, "batch"), (dict(batch=40000), -1, "batch"), (dict(next_n=0), -1, "next_n"), (dict(next_n=5), -1, "next_n"),
    (dict(num_heads=7), -1, "num_kv_heads"), (dict(num_kv_heads=0), -1, "num_kv_heads"),
    (dict(num_heads=260), -4, "128"), (dict(num_heads=128, next_n=4, num_kv_heads=2), -4, "128"),
    (dict(head_dim=96), -4, "head_dim"), (dict(head_dim=32), -4, "head_dim"),
    (dict(page_size=8), -1, "page_size"), (dict(page_size=48), -1, "page_size"),
    (dict(page_size=512), -1, "page_size"), (dict(num_pages=0), -1, "num_pages"),
    (dict(num_pages=2 ** 30), -4, "2^31"), (dict(max_pages_per_row=0), -1, "max_pages"),
    (dict(topk=-1), -1, "topk"), (dict(num_ctas=0), -1, "num_ctas"),
    (dict(num_ctas=5000), -1, "num_ctas"), (dict(dtype=2), -1, "dtype"), (dict(flags=4), -1, "flag"),
    (dict(q_stride_h=132), -1, "strides"), (dict(status=2), -1, "aligned"),
])
def test_bad_params(kw, code, needle):
    import ctypes
    lib, p = mq.library(), params(**kw)
    assert lib.paged_mqa_attention_fp4(16, 16, 16, 16, 16, 16, None, 16, None, 16, ctypes.byref(p), None) == code
    assert needle in lib.mqa_logits_last_error().decode()


@pytest.mark.parametrize("kw", [
    # a step past the end of what the kernels would walk does not fit an int32
    dict(max_pages_per_row=2 ** 23 - 1, page_size=256), dict(max_pages_per_row=2 ** 25 - 2 ** 10 + 1),
    dict(topk=2 ** 31 - 1), dict(topk=2 ** 31 - 2 ** 16 + 1)])
def test_lengths_that_would_wrap(kw):
    import ctypes
    lib, p, size = mq.library(), params(**kw), ctypes.c_uint64(0)
    assert lib.paged_mqa_attention_fp4(16, 16, 16, 16, 16, 16, 16, 16, None, 16, ctypes.byref(p), None) == -4
    assert "2147418112" in lib.mqa_logits_last_error().decode()
    assert lib.mqa_attention_workspace_size(ctypes.byref(p), ctypes.byref(size)) == -4


def test_rows_of_a_tile():
    """128 at most: all positions' heads on a kv head, or with lists one position's."""
    import ctypes
    lib, size = mq.library(), ctypes.c_uint64(0)
    for k, heads, n, fits in ((0, 64, 2, True), (0, 128, 2, False), (9, 128, 4, True), (9, 130, 1, False)):
        p = params(topk=k, num_heads=heads, next_n=n, num_kv_heads=1)
        rc = lib.mqa_attention_workspace_size(ctypes.byref(p), ctypes.byref(size))
        assert (rc == -4) == (not fits), (k, heads, n)  # without a GPU what fits stops at the device


def test_bad_pointers():
    import ctypes
    lib, p = mq.library(), params()
    good = [16, 16, 16, 16, 16, 16, None, 16, None, 16]
    for i in (0, 1, 2, 3, 4, 5, 7):
        args = list(good)
        args[i] = None
        assert lib.paged_mqa_attention_fp4(*args, ctypes.byref(p), None) == -1
        assert "NULL" in lib.mqa_logits_last_error().decode()
    for i, bad in ((0, 24), (1, 8), (2, 8), (3, 18), (4, 18), (5, 18), (7, 8), (8, 18), (9, 24)):
        args = list(good)
        args[i] = bad
        assert lib.paged_mqa_attention_fp4(*args, ctypes.byref(p), None) == -1
        assert "aligned" in lib.mqa_logits_last_error().decode()
    assert lib.paged_mqa_attention_fp4(*good, None, None) == -1
    lists = params(topk=8)
    assert lib.paged_mqa_attention_fp4(*good, ctypes.byref(lists), None) == -1
    assert "indices" in lib.mqa_logits_last_error().decode()
    assert lib.paged_mqa_attention_fp4(*[None] * 10, ctypes.byref(params(batch=0)), None) == 0
    size = ctypes.c_uint64(7)
    assert lib.mqa_attention_workspace_size(ctypes.byref(params(batch=0)), ctypes.byref(size)) == 0
    assert size.value == 0
    assert lib.mqa_attention_workspace_size(ctypes.byref(p), None) == -1


def test_params_struct_layout_matches_header():
    import ctypes
    assert ctypes.sizeof(mq.AttentionParams) == 96
    assert mq.AttentionParams.softmax_scale.offset == 48 and mq.AttentionParams.q_stride_b.offset == 56
    assert mq.AttentionParams.workspace_bytes.offset == 80 and mq.AttentionParams.status.offset == 88


def test_binding_checks_shapes():
    q = torch.zeros(2, 1, 8, 128, dtype=torch.bfloat16)
    kv = torch.zeros(4, 2 * 64 * 72, dtype=torch.uint8)
    bt, ctx = torch.zeros(2, 2, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    idx, sched = torch.zeros(2, 1, 4, dtype=torch.int32), torch.zeros(149, 2, dtype=torch.int32)

    def call(q=q, k=kv, v=kv, bt=bt, ctx=ctx, sched=sched, **kw):
        return mq.paged_mqa_attention_fp4(q, k, v, bt, ctx, sched, kv_heads=2, **kw)

    with pytest.raises(ValueError, match="q must be"):
        call(q=q[0])
    with pytest.raises(ValueError, match="either"):
        call(indices=idx)
    with pytest.raises(ValueError, match="either"):
        call(sched=None)
    with pytest.raises(ValueError, match="dtype"):
        call(q=q.float())
    with pytest.raises(ValueError, match="contiguous"):
        call(q=q.transpose(2, 3).contiguous().transpose(2, 3))
    with pytest.raises(ValueError, match="differ"):
        call(v=kv[:3])
    with pytest.raises(ValueError, match="pages hold"):
        call(page_size=32)
    with pytest.raises(ValueError, match="indices must"):
        call(sched=None, indices=idx[:1])
    with pytest.raises(ValueError, match="at least one"):
        call(sched=None, indices=idx[:, :, :0])
    with pytest.raises(ValueError, match="CUDA"):
        call()  # host tensors: no CPU path

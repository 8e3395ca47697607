"""The 4-bit key/value cache on the GPU against ``cachelib``: what append
writes and read returns bit for bit, attention within the bound of its
roundings, errors, streams and graphs, and a round of attention, verification
and append together."""
import math

import numpy as np
import pytest
import torch

import draft_token_verification_verify_b200 as sv
from cachelib import TYPES, Pages, attention, paths, quantise

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _device(cuda_device):
    import __graft_entry__

    __graft_entry__.build()
    return cuda_device


def gen(seed):
    return torch.Generator().manual_seed(seed)


def dev(t):
    return t.to("cuda:0")


class Case:
    """A cache with random contents and B sequences of the given lengths."""

    def __init__(self, lens, page, heads, D, T, n, seed=0, spare=2, fill=True):
        g = gen(seed)
        need = [-(-(max(x, 0) + n) // page) for x in lens]
        self.pages = Pages(sum(need) + spare, heads, page, D, T)
        if fill:
            self.pages.random(g)
        ids = torch.randperm(sum(need) + spare, generator=g)
        self.table = torch.full((len(lens), max(need)), -5, dtype=torch.int32)
        at = 0
        for b, m in enumerate(need):
            self.table[b, :m] = ids[at:at + m].int()
            at += m
        self.lens, self.page, self.heads, self.D, self.T, self.n = list(lens), page, heads, D, T, n
        self.g = g
        self.raw = dev(self.pages.bytes())
        self.cache = sv.KvCache(self.raw, D, T)
        self.d_table, self.d_lens = dev(self.table), dev(torch.tensor(lens, dtype=torch.int32))

    def tokens(self, heads, sigma=1.0):
        return (sigma * torch.randn((len(self.lens), self.n, heads, self.D), generator=self.g)).to(self.T)

    def want(self, q, k=None, v=None, parents=None, scale=None):
        """(out, lse, tolerance) in 64 bits, stacked over the sequences."""
        scale = self.D ** -0.5 if scale is None else scale
        got = []
        for b, m in enumerate(self.lens):
            m = max(m, 0)
            kc, _ = self.pages.rows(0, self.table[b], m)
            vc, vs = self.pages.rows(1, self.table[b], m)
            see = torch.ones((self.n, m), dtype=torch.bool)
            if k is not None:
                kc, vc = torch.cat((kc, k[b].double())), torch.cat((vc, v[b].double()))
                vs = torch.cat((vs, torch.zeros((self.n, self.heads), dtype=torch.float64)))
                see = torch.cat((see, paths(self.n, None if parents is None else parents[b])), 1)
            got.append(attention(q[b], kc, vc, vs, see, scale, self.T))
        return [torch.stack(x) for x in zip(*got)]

    def attend(self, q, k=None, v=None, parents=None, **kw):
        lse = torch.full(q.shape[:3], 7.0, dtype=torch.float32, device="cuda:0")
        out = sv.cache_attend(dev(q), self.cache, self.d_table, self.d_lens, None if k is None else dev(k),
                              None if v is None else dev(v), parents=None if parents is None else dev(parents),
                              out_lse=lse, **kw)
        torch.cuda.synchronize()
        return out.cpu().double(), lse.cpu().double()


def check(got, lse, want):
    out, ref_lse, tol = want
    off = (got - out).abs()
    assert bool((off <= tol).all()), f"off by {float((off / tol).max()):.3g} of the bound"
    empty = ref_lse == -math.inf
    assert bool((lse[empty] == -math.inf).all())
    np.testing.assert_allclose(lse[~empty].numpy(), ref_lse[~empty].numpy(), rtol=1e-4, atol=1e-4)


SHAPES = [  # lens, page, kv heads, group, D, n
    ([1], 16, 1, 1, 64, 1),
    ([0], 64, 2, 4, 128, 1),
    ([63, 64, 65], 64, 1, 4, 128, 2),
    ([15, 16, 17, 0, 31], 16, 2, 3, 64, 5),
    ([100, 33, 7], 32, 3, 5, 128, 3),
    ([257, 128, 640], 128, 2, 8, 128, 9),
    ([1000, 0, -1, 999], 1024, 1, 7, 128, 4),
    ([5000], 64, 1, 1, 128, 1),
    ([3001, 12, 2048, 700], 32, 4, 2, 64, 17),
    ([40, 90], 16, 1, 16, 128, 20),
    ([500], 64, 2, 1, 128, 257),
]


@pytest.mark.parametrize("kind", ["bf16", "fp16"])
@pytest.mark.parametrize("alone", [False, True])
@pytest.mark.parametrize("lens,page,heads,group,D,n", SHAPES)
def test_attend(lens, page, heads, group, D, n, alone, kind):
    c = Case(lens, page, heads, D, TYPES[kind], n, seed=n + D)
    q, k, v = c.tokens(heads * group, 1.5), c.tokens(heads), c.tokens(heads)
    if alone:
        check(*c.attend(q), c.want(q))
    else:
        check(*c.attend(q, k, v), c.want(q, k, v))


TREES = {
    "binary": lambda n: np.arange(n - 1) // 2,
    "star": lambda n: np.zeros(n - 1, int),
    "late": lambda n: np.maximum(np.arange(n - 1) - 3, 0),
}


@pytest.mark.parametrize("kind", ["bf16", "fp16"])
@pytest.mark.parametrize("shape", list(TREES))
@pytest.mark.parametrize("n,group,D", [(2, 1, 64), (9, 4, 128), (18, 2, 64), (33, 8, 128), (66, 1, 128), (257, 1, 64)])
def test_attend_tree(n, group, D, shape, kind):
    lens = [130, 0, 70]
    c = Case(lens, 32, 2, D, TYPES[kind], n, seed=n)
    par = torch.tensor(np.tile(TREES[shape](n), (3, 1)), dtype=torch.int32)
    if n > 4:
        par[1] = torch.arange(n - 1, dtype=torch.int32)  # a chain beside the trees
    q, k, v = c.tokens(2 * group, 1.5), c.tokens(2), c.tokens(2)
    check(*c.attend(q, k, v, par), c.want(q, k, v, par))


def test_attend_chain_equals_its_tree():
    c = Case([300, 64], 64, 2, 128, torch.bfloat16, 6, seed=3)
    q, k, v = c.tokens(8), c.tokens(2), c.tokens(2)
    par = torch.arange(5, dtype=torch.int32).repeat(2, 1)
    a, b = c.attend(q, k, v), c.attend(q, k, v, par)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("n,group", [(1, 4), (5, 4), (9, 8)])
def test_attend_long_split(n, group):
    """A context cut over the whole device, beside a short one; the same bits every time."""
    c = Case([30011, 5], 64, 2, 128, torch.bfloat16, n, seed=7)
    q, k, v = c.tokens(2 * group, 1.5), c.tokens(2), c.tokens(2)
    a = c.attend(q, k, v)
    check(*a, c.want(q, k, v))
    b = c.attend(q, k, v)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_attend_many_sequences():
    """More segments than CTAs, and more sequences than a CTA has threads."""
    lens = [(b * 37) % 200 for b in range(400)]
    c = Case(lens, 16, 2, 64, torch.bfloat16, 2, seed=11)
    q, k, v = c.tokens(4), c.tokens(2), c.tokens(2)
    check(*c.attend(q, k, v), c.want(q, k, v))


@pytest.mark.parametrize("D,cap", [(64, 0), (64, 1100), (128, 0)])
def test_attend_more_sequences_than_threads(D, cap):
    """Short contexts of so many sequences that the warps take ranges of them, whole segments among them; two
    sequences a thread in the search for a range's first.  Some have no tokens or are no sequences."""
    lens = [(b * 37) % 150 if b % 11 else -(b % 2) for b in range(300)]
    c = Case(lens, 16, 5, D, torch.bfloat16, 3, seed=37)
    if cap:
        c.d_table = torch.cat((c.d_table, torch.zeros((300, cap // 16), dtype=torch.int32, device="cuda:0")), 1)
    q, k, v = c.tokens(10), c.tokens(5), c.tokens(5)
    check(*c.attend(q, k, v), c.want(q, k, v))
    check(*c.attend(q), c.want(q))


@pytest.mark.parametrize("n,group,D,lens", [(65, 16, 64, [1100, 40]), (129, 5, 128, [1300]), (33, 33, 128, [20, 2000])])
def test_attend_more_rows_than_one_pass(n, group, D, lens):
    """More row blocks than go side by side, the last of them not full; contexts that are cut."""
    c = Case(lens, 64, 2, D, torch.bfloat16, n, seed=41)
    q, k, v = c.tokens(2 * group, 1.5), c.tokens(2), c.tokens(2)
    check(*c.attend(q, k, v), c.want(q, k, v))
    par = torch.tensor(np.tile(TREES["binary"](n), (len(lens), 1)), dtype=torch.int32)
    check(*c.attend(q, k, v, par), c.want(q, k, v, par))


def test_cut_and_whole_segments_agree():
    """The form for few short contexts against the one that cuts them: the same attention."""
    for D in (64, 128):
        c = Case([700, 3, 0, 450], 64, 2, D, torch.bfloat16, 5, seed=43)
        q, k, v = c.tokens(8, 1.5), c.tokens(2), c.tokens(2)
        want = c.want(q, k, v)
        st = torch.full((1,), 5, dtype=torch.int32, device="cuda:0")
        check(*c.attend(q, k, v), want)
        check(*c.attend(q, k, v, out_status=st), want)
        assert st.item() == sv.SV_OK


@pytest.mark.parametrize("lens", [[300, 70], [3000, 70]])
@pytest.mark.parametrize("D", [64, 128])
def test_attend_magnitudes(D, lens):
    """Powers of two on the keys (and their inverse on the queries) and on the values change no rounding: the
    same bits times the values' power, over the range that is documented."""
    T = torch.bfloat16
    first = None
    for ek, ev in ((0, 0), (-55, 0), (55, 0), (0, -60), (0, 52), (30, -30)):
        c = Case(lens, 64, 2, D, T, 3, seed=59)
        for part, e in ((0, ek), (1, ev)):
            c.pages.params[part] = (c.pages.params[part].double() * 2.0 ** e).to(T)
        c.raw.copy_(c.pages.bytes())
        q, k, v = (x.double() for x in (c.tokens(8, 1.5), c.tokens(2), c.tokens(2)))
        out, lse = c.attend((q * 2.0 ** -ek).to(T), (k * 2.0 ** ek).to(T), (v * 2.0 ** ev).to(T))
        if first is None:
            first = out, lse
        assert torch.equal(lse, first[1]), (ek, ev)
        if ev > -50:
            assert torch.equal(out, first[0] * 2.0 ** ev), (ek, ev)
        else:
            # a weight of a long context times 2^-60 and a code's 2^-133 lies among fp32's subnormals: each of at
            # most as many additions as tokens is off by half their spacing, 2^-150, which the output's 2^69
            # makes 2^-81 (the sum of weights it is divided by is at least 1), for the sum and the one of 8 each;
            # where that crosses a rounding to bf16, one step, 2^-7 of the output, more
            off = (out - first[0] * 2.0 ** ev).abs()
            assert bool((off <= 2.0 ** -7 * out.abs() + 2 * (max(lens) + 3) * 2.0 ** -81).all()), (ek, ev)


def test_pages_past_4_gib():
    """Pages whose offset passes 32 bits: appended to, read and attended as the same pages of a small cache."""
    c = Case([130], 64, 8, 128, torch.bfloat16, 4, seed=47)
    q, k, v = c.tokens(32), c.tokens(8), c.tokens(8)
    num = 64000  # of 69,632 bytes
    far = torch.empty((num, *c.raw.shape[1:]), dtype=torch.uint8, device="cuda:0")
    at = torch.tensor([num - 1 - 7 * i for i in range(c.raw.shape[0])], device="cuda:0")
    far[at] = c.raw
    big, table = sv.KvCache(far, 128), at[c.d_table.long()].int()
    outs = []
    for cache, t in ((c.cache, c.d_table), (big, table)):
        o = sv.cache_attend(dev(q), cache, t, c.d_lens, dev(k), dev(v))
        lens = sv.cache_append(cache, t, c.d_lens, dev(k), dev(v))
        outs.append((o, lens) + sv.cache_read(cache, t, lens, 134))
    for a, b in zip(*outs):
        assert torch.equal(a, b)
    assert torch.equal(far[at], c.raw)


def test_two_graphs_replayed_side_by_side():
    """A step of attention, append and read captured twice, each with its own workspace, on two streams."""
    steps = []
    for i in range(2):
        c = Case([1500, 40 + i, 0], 64, 2, 128, torch.bfloat16, 3, seed=51 + i)
        q, k, v = c.tokens(8), c.tokens(2), c.tokens(2)
        want = c.want(q, k, v)
        d = [dev(x) for x in (q, k, v)]
        ws = torch.empty(c.cache.workspace_bytes(3, 3, 8), dtype=torch.uint8, device="cuda:0")
        out, new = torch.empty_like(d[0]), torch.empty(3, dtype=torch.int32, device="cuda:0")
        rk, rv = (torch.empty((3, 3, 2, 128), dtype=torch.bfloat16, device="cuda:0") for _ in range(2))

        def step(c=c, d=d, ws=ws, out=out, new=new, rk=rk, rv=rv):
            sv.cache_attend(d[0], c.cache, c.d_table, c.d_lens, d[1], d[2], out=out, workspace=ws)
            sv.cache_append(c.cache, c.d_table, c.d_lens, d[1], d[2], out_lens=new)
            sv.cache_read(c.cache, c.d_table, new, 3, first=c.d_lens, out_k=rk, out_v=rv)

        step()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step()
        # (with the step, which holds the inputs and the workspace that the graph goes on using)
        steps.append((c, g, k, v, want, out, new, rk, rv, step, torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(5):
        for s in steps:
            s[5].zero_()
        torch.cuda.synchronize()
        for s in steps:
            with torch.cuda.stream(s[-1]):
                s[1].replay()
    torch.cuda.synchronize()
    for c, _, k, v, want, out, new, rk, rv, _, _ in steps:
        assert bool(((out.cpu().double() - want[0]).abs() <= want[2]).all())
        assert new.tolist() == [x + 3 for x in c.lens]
        for x, got in ((k, rk), (v, rv)):
            codes, scale, zero = quantise(x)
            assert torch.equal(got.cpu(), (zero.double()[..., None] + scale.double()[..., None] * codes.double()).to(c.T))


def test_attend_scale_and_large_scores():
    """Scores far apart: the running maximum moves by more than the threshold, early and late."""
    c = Case([700, 700], 64, 1, 128, torch.bfloat16, 2, seed=5)
    q, k, v = c.tokens(4, 6.0), c.tokens(1), c.tokens(1)
    for scale in (0.5, 2.0, -0.25, 0.0):
        out, lse = c.attend(q, k, v, scale=scale)
        want = c.want(q, k, v, scale=scale)
        # the scores' fp32 error grows with their size
        assert bool(((out - want[0]).abs() <= want[2] + 0.02 * abs(scale)).all())
        np.testing.assert_allclose(lse.numpy(), want[1].numpy(), rtol=1e-4, atol=1e-2)


def test_attend_strided_projection_rows():
    """q, k and v as parts of one fused projection's rows."""
    c = Case([90, 200], 64, 2, 64, torch.float16, 3, seed=9)
    rows = torch.randn((2, 3, 12, 64), generator=c.g).half()
    q, k, v = rows[:, :, :8], rows[:, :, 8:10], rows[:, :, 10:]
    d = dev(rows)
    out = sv.cache_attend(d[:, :, :8], c.cache, c.d_table, c.d_lens, d[:, :, 8:10], d[:, :, 10:])
    assert torch.equal(out.cpu().double(), c.attend(q.contiguous(), k.contiguous(), v.contiguous())[0])


def test_attend_ignores_what_is_not_seen():
    """NaN and infinities behind the lengths, in other branches and in later drafts reach no one."""
    n, par = 5, torch.tensor([[0, 0, 1, 2]], dtype=torch.int32)
    for T in (torch.bfloat16, torch.float16):
        c = Case([70], 32, 2, 128, T, n, seed=13)
        c.pages.params[0][c.table[0, 2], :, 6:] = math.nan  # tokens 70 and up
        c.pages.params[1][c.table[0, 2], :, 6:] = math.inf
        c.cache.pages.copy_(dev(c.pages.bytes()))
        q, k, v = c.tokens(8), c.tokens(2), c.tokens(2)
        clean = c.want(q, k, v, par)
        k2, v2 = k.clone(), v.clone()
        k2[0, 3], v2[0, 3] = math.nan, math.nan   # node 3: below node 1, seen by itself alone
        v2[0, 4, :, 7], k2[0, 4, :, 3] = math.inf, -math.inf
        out, lse = c.attend(q, k2, v2, par)
        for i in (0, 1, 2):
            assert bool(((out[0, i] - clean[0][0, i]).abs() <= clean[2][0, i]).all())
        assert bool(torch.isnan(out[0, 3]).all())
        # the chain: nodes before a value with an infinity
        out, _ = c.attend(q, k, v2)
        ref = c.want(q, k, v)
        assert bool(((out[0, :3] - ref[0][0, :3]).abs() <= ref[2][0, :3]).all())
        assert bool(torch.isnan(out[0, 3:]).any(-1).all())


def test_attend_cached_nan_is_loud():
    c = Case([70, 70], 32, 1, 64, torch.bfloat16, 1, seed=15)
    c.pages.params[1][c.table[0, 1], 0, 3] = math.nan
    c.cache.pages.copy_(dev(c.pages.bytes()))
    q = c.tokens(2)
    out, _ = c.attend(q)
    want = c.want(q)
    assert bool(torch.isnan(out[0]).all())
    assert bool(((out[1] - want[0][1]).abs() <= want[2][1]).all())


def test_attend_data_errors():
    """A page out of range, a length above the table, a parent out of range: that sequence is NaN, the others right."""
    c = Case([100, 100, 100, 100], 32, 2, 64, torch.bfloat16, 3, seed=17)
    q, k, v = c.tokens(4), c.tokens(2), c.tokens(2)
    par = torch.tensor([[0, 1]] * 4, dtype=torch.int32)
    want = c.want(q, k, v, par)
    c.d_table[0, 1] = c.pages.num
    c.d_lens[1] = c.table.shape[1] * 32 + 1
    bad = par.clone()
    bad[2, 1] = 2  # node 2 its own parent
    out, _ = c.attend(q, k, v, bad)
    for b in range(3):
        assert bool(torch.isnan(out[b]).all()), b
    assert bool(((out[3] - want[0][3]).abs() <= want[2][3]).all())
    c.d_table[0, 1] = -1
    bad[2, 1] = -1
    out, _ = c.attend(q, k, v, bad)
    assert bool(torch.isnan(out[:3]).all())


@pytest.mark.parametrize("page,fill", [(64, 0), (64, 30), (16, 0), (16, 30)])
def test_attend_bad_pages_of_few_sequences(page, fill):
    """Every tenth sequence is long, the rest leave some warps without a cached tile: a bad page of one of
    them, far ahead of the segment that is computed, is that sequence's alone."""
    lens = [290 if b % 10 == 9 else fill for b in range(70)] + [3000]
    c = Case(lens, page, 2, 64, torch.bfloat16, 64, seed=31)
    q, k, v = c.tokens(16), c.tokens(2), c.tokens(2)
    want = c.want(q, k, v)
    bad = [9, 29, 39, 49, 69]
    for i, b in enumerate(bad):
        c.d_table[b, (64 * (3 - i % 4) + 63) // page] = -1 if i % 2 else c.pages.num
    out, lse = c.attend(q, k, v)
    fine = ((out - want[0]).abs() <= want[2]).all(-1).all(-1).all(-1)
    for b in range(len(lens)):
        if b in bad:
            assert bool(torch.isnan(out[b]).all()) and bool(torch.isnan(lse[b]).all()), b
        else:
            assert bool(fine[b]), b


def test_attend_wait_that_runs_out():
    c = Case([200], 64, 1, 128, torch.bfloat16, 2, seed=19)
    q = c.tokens(4)
    st = torch.full((1,), 5, dtype=torch.int32, device="cuda:0")
    out, _ = c.attend(q, opts=sv.make_options(test_extra_tx=16, wait_timeout_ns=1_000_000), out_status=st)
    assert st.item() == sv.SV_ERR_DEVICE_TIMEOUT and bool(torch.isnan(out).all())
    out, lse = c.attend(q, out_status=st)
    assert st.item() == sv.SV_OK
    check(out, lse, c.want(q))


def test_attend_graph_replays_with_new_lengths():
    """Captured once, replayed as the lengths grow: nothing of a length is kept on the host."""
    c = Case([10, 300], 32, 2, 64, torch.bfloat16, 2, seed=21)
    q, k, v = c.tokens(4), c.tokens(2), c.tokens(2)
    d = [dev(x) for x in (q, k, v)]
    ws = torch.empty(sv.spec_cache_attend_workspace_size(2, 2, 4, 2, 64), dtype=torch.uint8, device="cuda:0")
    out = torch.empty_like(d[0])
    lens = torch.tensor([3, 1], dtype=torch.int32, device="cuda:0")
    sv.cache_attend(d[0], c.cache, c.d_table, lens, d[1], d[2], out=out, workspace=ws)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        sv.cache_attend(d[0], c.cache, c.d_table, lens, d[1], d[2], out=out, workspace=ws)
    for new in ([3, 1], [10, 300], [0, 64]):
        lens.copy_(torch.tensor(new, dtype=torch.int32))
        g.replay()
        torch.cuda.synchronize()
        c.lens = new
        want = c.want(q, k, v)
        assert bool(((out.cpu().double() - want[0]).abs() <= want[2]).all())


def test_attend_two_streams():
    c = Case([4000, 900], 64, 2, 128, torch.bfloat16, 3, seed=23)
    q, k, v = c.tokens(8), c.tokens(2), c.tokens(2)
    d = [dev(x) for x in (q, k, v)]
    want = c.want(q, k, v)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [sv.cache_attend(d[0], c.cache, c.d_table, c.d_lens, d[1], d[2], stream=streams[i % 2]) for i in range(8)]
    torch.cuda.synchronize()
    for o in outs:
        assert bool(((o.cpu().double() - want[0]).abs() <= want[2]).all())
    raw = sv.cache_attend(d[0], c.cache, c.d_table, c.d_lens, d[1], d[2], stream=streams[0].cuda_stream)
    torch.cuda.synchronize()
    assert torch.equal(raw, outs[0])


# ---- append and read ------------------------------------------------------------------

def append(c, k, v, **kw):
    lens = sv.cache_append(c.cache, c.d_table, c.d_lens, dev(k), dev(v), **kw)
    torch.cuda.synchronize()
    return lens


def expect_append(c, k, v, rows):
    """The pages after sequence b kept its rows[b] (list of nodes)."""
    for b, nodes in enumerate(rows):
        for i, node in enumerate(nodes):
            pos = c.lens[b] + i
            page, at = int(c.table[b, pos // c.page]), pos % c.page
            c.pages.put(0, page, at, k[b, node])
            c.pages.put(1, page, at, v[b, node])


def same_pages(c):
    want = c.pages.bytes()
    got = c.raw.cpu()
    if torch.equal(got, want):
        return
    g = Pages.of(got, c.page, c.D, c.T)
    for i in range(2):
        assert torch.equal(g.codes[i], c.pages.codes[i]), f"codes of {'kv'[i]}: " \
            f"{int((g.codes[i] != c.pages.codes[i]).sum())} differ"
        a, b = g.params[i].view(torch.int16), c.pages.params[i].view(torch.int16)
        nan = torch.isnan(g.params[i]) & torch.isnan(c.pages.params[i])
        zero = (g.params[i] == 0) & (c.pages.params[i] == 0)
        assert bool(((a == b) | nan | zero).all()), "parameters"


@pytest.mark.parametrize("kind", ["bf16", "fp16"])
@pytest.mark.parametrize("lens,page,heads,D,n", [
    ([0], 16, 1, 64, 1), ([0, 63, 64, 65], 64, 2, 128, 9), ([5, 14, 31], 16, 3, 64, 40), ([7, 100], 32, 5, 128, 3),
    ([0, 200], 128, 2, 128, 300), ([1000], 1024, 1, 64, 70),
])
def test_append_writes_the_definition(lens, page, heads, D, n, kind):
    c = Case(lens, page, heads, D, TYPES[kind], n, seed=n)
    k, v = c.tokens(heads, 2.0) + 1, c.tokens(heads)
    new = append(c, k, v)
    assert new.tolist() == [x + n for x in lens]
    expect_append(c, k, v, [range(n)] * len(lens))
    same_pages(c)


def test_append_counts_nodes_and_inactive():
    lens = [20, 3, 0, 7, -1, 40]
    c = Case(lens, 16, 2, 64, torch.bfloat16, 6, seed=2)
    k, v = c.tokens(2), c.tokens(2)
    acc = torch.tensor([5, 0, -1, 2, 3, 1], dtype=torch.int32)
    nodes = torch.full((6, 6), -1, dtype=torch.int32)
    nodes[0, :5] = torch.tensor([1, 2, 3, 4, 5])
    nodes[3, :2] = torch.tensor([2, 5])
    nodes[5, :1] = 3
    new = append(c, k, v, n_accepted=dev(acc), nodes=dev(nodes))
    assert new.tolist() == [26, 4, 0, 10, -1, 42]
    expect_append(c, k, v, [[0, 1, 2, 3, 4, 5], [0], [], [0, 2, 5], [], [0, 3]])
    same_pages(c)


def test_append_in_place_step_by_step():
    """One and two tokens at a time, the lengths advanced in place: the same pages as in one go."""
    c = Case([0, 13], 16, 2, 128, torch.bfloat16, 40, seed=4)
    k, v = c.tokens(2), c.tokens(2)
    at = 0
    for m in (1, 2, 1, 3, 8, 1, 9, 15):
        out = sv.cache_append(c.cache, c.d_table, c.d_lens, dev(k[:, at:at + m].contiguous()),
                              dev(v[:, at:at + m].contiguous()), out_lens=c.d_lens)
        assert out is c.d_lens
        at += m
    torch.cuda.synchronize()
    assert at == 40 and c.d_lens.tolist() == [40, 53]
    expect_append(c, k, v, [range(40)] * 2)
    same_pages(c)


@pytest.mark.parametrize("kind", ["bf16", "fp16"])
def test_append_hard_rows(kind):
    """Constant rows, ties, one outlier, the smallest and largest magnitudes, NaN and infinities."""
    T = TYPES[kind]
    info = torch.finfo(T)
    D, n = 64, 16
    c = Case([0], 16, 1, D, T, n, seed=6)
    k = torch.zeros((1, n, 1, D), dtype=T)
    k[0, 0] = 3.0
    k[0, 1, 0] = torch.arange(D).to(T) / 2           # exact halves of a step: ties to even
    k[0, 2, 0, :2] = torch.tensor([0.0, 15.0]).to(T)
    k[0, 2, 0, 2:33] = torch.arange(31).to(T) / 2    # 0, .5, 1, ... 15 at scale 1
    k[0, 3, 0, 5] = 1000.0
    k[0, 4, 0, 1] = info.smallest_normal
    k[0, 5, 0, 1] = info.smallest_normal * info.eps  # the smallest subnormal
    k[0, 6, 0, ::2] = info.max / 4
    k[0, 6, 0, 1::2] = -info.max / 4
    k[0, 7, 0] = -0.0
    k[0, 8, 0, 9] = math.nan
    k[0, 9, 0, 9] = math.inf
    k[0, 10, 0, 9] = -math.inf
    k[0, 11, 0, 0], k[0, 11, 0, 1] = info.max, -info.max  # a range beyond the type, or not
    k[0, 12, 0] = (torch.arange(D) % 31).to(T) * 3 - 40
    k[0, 13, 0] = torch.randn(D, generator=c.g).to(T) * info.smallest_normal * 20
    k[0, 14, 0] = torch.randn(D, generator=c.g).to(T)
    k[0, 15, 0] = torch.randn(D, generator=c.g).to(T) * 1e3 + 5e3
    v = k.flip(1).contiguous()
    append(c, k, v)
    expect_append(c, k, v, [range(n)])
    same_pages(c)
    rk, _ = sv.cache_read(c.cache, c.d_table, dev(torch.tensor([n], dtype=torch.int32)), n)
    rk = rk.cpu()
    assert bool(torch.isnan(rk[0, 8:11]).all()) and bool((rk[0, 0] == 3.0).all())


@pytest.mark.parametrize("kind", ["bf16", "fp16"])
@pytest.mark.parametrize("D", [64, 128])
def test_append_halves(kind, D):
    """Quotients on a half, and as close to one as the types allow (a half less or more a number that is tiny
    beside the row's minimum), over scales of every mantissa."""
    T = TYPES[kind]
    n = 512
    c = Case([3], 64, 2, D, T, n, seed=8)
    x = torch.zeros((n, 2, D), dtype=torch.float64)
    for r in range(n):
        s = (128 + r % 128) * 2.0 ** (-9 - (r // 128) % 2)
        x[r, 0] = torch.randint(0, 31, (D,), generator=c.g).double() / 2 * s
        x[r, 0, :2] = torch.tensor([0.0, 15 * s])
        zero = -0.5 * s if r % 3 == 0 else -1.5 * s if r % 3 == 1 else -7.5 * s
        tiny = torch.randint(-8, 9, (D,), generator=c.g).double() * s * 2.0 ** -(20 + r % 7 if T == torch.bfloat16 else 10 + r % 4)
        x[r, 1] = torch.where(torch.rand(D, generator=c.g) < 0.7, tiny, zero + torch.randint(0, 31, (D,), generator=c.g) / 2 * s)
        x[r, 1, :2] = torch.tensor([zero, zero + 15 * s])
    k = x[None].to(T)
    v = k.flip(1).contiguous()
    append(c, k, v)
    expect_append(c, k, v, [range(n)])
    same_pages(c)


def test_append_data_errors():
    lens = [20, 20, 20, 44, 20]
    c = Case(lens, 16, 2, 64, torch.bfloat16, 5, seed=8)
    c.d_table[1, 1] = c.pages.num + 3
    k, v = c.tokens(2), c.tokens(2)
    acc = torch.tensor([4, 4, 5, 4, 4], dtype=torch.int32)  # sequence 2: more rows than there are
    nodes = torch.arange(1, 6, dtype=torch.int32).repeat(5, 1)
    nodes[4, 1] = 5  # no such node
    new = append(c, k, v, n_accepted=dev(acc), nodes=dev(nodes))
    assert c.table.shape[1] * 16 == 64 and new.tolist() == [25, -1, -1, 49, -1]
    # earlier tokens of the failed sequences, and everyone else's, are untouched
    got = Pages.of(c.raw, 16, 64, c.T)
    expect_append(c, k, v, [range(5), [], [], range(5), []])
    for b in range(5):
        m = lens[b] + (5 if b in (0, 3) else 0)
        if b != 1:
            for i in range(2):
                assert torch.equal(got.rows(i, c.table[b], m)[0], c.pages.rows(i, c.table[b], m)[0])
    c2 = Case([60], 16, 1, 64, torch.bfloat16, 3, seed=8)  # 64 mapped tokens
    c2.d_lens[0] = 62
    assert append(c2, c2.tokens(1), c2.tokens(1)).tolist() == [-1]
    c2.d_lens[0] = 61
    assert append(c2, c2.tokens(1), c2.tokens(1)).tolist() == [64]


@pytest.mark.parametrize("kind", ["bf16", "fp16"])
@pytest.mark.parametrize("page,D,heads,n,first", [
    (16, 64, 3, 50, None), (64, 128, 2, 7, [0, 60, 195]), (128, 128, 1, 260, [-3, 100, 1]), (32, 64, 1, 1, [31, 32, 199]),
])
def test_read(page, D, heads, n, first, kind):
    lens = [70, -1, 200]
    c = Case(lens, page, heads, D, TYPES[kind], 1, seed=page)
    f = None if first is None else dev(torch.tensor(first, dtype=torch.int32))
    k, v = sv.cache_read(c.cache, c.d_table, c.d_lens, n, first=f)
    for part, got in enumerate((k.cpu(), v.cpu())):
        for b, m in enumerate(lens):
            want = torch.zeros((n, heads, D), dtype=c.T)
            all_rows = c.pages.rows(part, c.table[b], max(m, 0))[0].float().to(c.T)
            for i in range(n):
                pos = i + (first[b] if first else 0)
                if 0 <= pos < m:
                    want[i] = all_rows[pos]
            assert torch.equal(got[b], want)


def test_read_bad_pages_are_nan():
    c = Case([70, 70], 32, 2, 64, torch.bfloat16, 1, seed=3)
    c.d_table[0, 1] = -1
    c.d_lens[1] = 200  # the table ends at 96
    k, v = sv.cache_read(c.cache, c.d_table, c.d_lens, 110)
    for x in (k.cpu(), v.cpu()):
        assert bool(torch.isnan(x[0, 32:64]).all()) and not bool(torch.isnan(x[0, :32]).any())
        assert not bool(torch.isnan(x[0, 64:]).any()) and not bool(torch.isnan(x[1, :96]).any())
        assert bool(torch.isnan(x[1, 96:]).all())


# ---- a round: attention, verification, append --------------------------------------------

@pytest.mark.parametrize("tree", [False, True])
def test_round(tree):
    """Two rounds of one attention layer over the cache with its own verification: the cache that append
    leaves, and the attention of the next round over it, equal those of a cache written by hand."""
    B, n, heads, group, D, V = 3, 7, 2, 4, 64, 50
    c = Case([40, 0, 93], 16, heads, D, torch.bfloat16, 2 * n, seed=31)
    c.n = n
    g = c.g
    head = torch.randn((V, heads * group * D), generator=g) / 4
    par = torch.tensor([[0, 0, 1, 1, 2, 4]] * B, dtype=torch.int32) if tree else None
    for step in range(2):
        q, k, v = c.tokens(heads * group, 1.5), c.tokens(heads), c.tokens(heads)
        out = sv.cache_attend(dev(q), c.cache, c.d_table, c.d_lens, dev(k), dev(v), parents=None if par is None else dev(par))
        want = c.want(q, k, v, par)
        assert bool(((out.cpu().double() - want[0]).abs() <= want[2]).all())
        logits = (out.float().reshape(B, n, -1) @ dev(head).T).contiguous()
        toks = logits.argmax(-1)[:, :n - 1].int()          # of its parent in a chain: drafts that pass ...
        if tree:
            toks = logits.argmax(-1).gather(1, dev(par).long()).int()
        toks[0, 2] = (toks[0, 2] + 1) % V                   # ... but for a few
        toks[1, 0] = (toks[1, 0] + 1) % V
        toks = toks.contiguous()
        if tree:
            nodes = torch.empty((B, n), dtype=torch.int32, device="cuda:0")
            _, acc = sv.verify_tree(logits, None, toks, dev(par), greedy=True, out_nodes=nodes)
        else:
            nodes = None
            _, acc = sv.verify(logits, None, toks, greedy=True)
        new = sv.cache_append(c.cache, c.d_table, c.d_lens, dev(k), dev(v), n_accepted=acc, nodes=nodes)
        torch.cuda.synchronize()
        rows = []
        for b in range(B):
            m = int(acc[b])
            assert m >= 0
            rows.append([0] + ([int(i) for i in nodes[b, :m]] if tree else list(range(1, m + 1))))
        assert max(len(r) for r in rows) > 2
        expect_append(c, k, v, rows)
        same_pages(c)
        c.lens = [a + len(r) for a, r in zip(c.lens, rows)]
        assert new.tolist() == c.lens
        c.d_lens = new


def test_round_in_a_graph():
    """Attention and an in-place append captured together and replayed: the lengths live on the device."""
    c = Case([5, 30], 16, 1, 64, torch.bfloat16, 12, seed=33)
    c.n = 2
    q, k, v = (c.tokens(h) for h in (4, 1, 1))
    d = [dev(x) for x in (q, k, v)]
    acc = torch.tensor([1, 0], dtype=torch.int32, device="cuda:0")
    ws = torch.empty(sv.spec_cache_attend_workspace_size(2, 2, 4, 1, 64), dtype=torch.uint8, device="cuda:0")
    out = torch.empty_like(d[0])

    def step():
        sv.cache_attend(d[0], c.cache, c.d_table, c.d_lens, d[1], d[2], out=out, workspace=ws)
        sv.cache_append(c.cache, c.d_table, c.d_lens, d[1], d[2], n_accepted=acc, out_lens=c.d_lens)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        step()
    torch.cuda.synchronize()
    for _ in range(4):
        want = c.want(q, k, v)
        g.replay()
        torch.cuda.synchronize()
        assert bool(((out.cpu().double() - want[0]).abs() <= want[2]).all())
        expect_append(c, k, v, [[0, 1], [0]])
        same_pages(c)
        c.lens = [c.lens[0] + 2, c.lens[1] + 1]
        assert c.d_lens.tolist() == c.lens

"""Page keys and page-selected decode.

Keys, scales and selected pages have a defined value (each step one fp32
operation, the sums exact), so they are compared bit for bit with the same steps
on the CPU.  The attention over the selected pages is compared with fp64:
probabilities enter the second product as bf16 (2^-8 of each) and the output is
rounded to bf16 (2^-8 of it), so |o - o64| <= 2^-8 (A + |o64|) with
A = sum_i p_i |v_i|; SCORE bounds the relative error of a probability from the
fp32 scores (independent roundings: sqrt(576) * 2^-24 * 40 < 2^-13) and the
absolute error of the LSE.
"""
import math

import pytest
import torch

from mla_paged_kv_03_b200 import binding as B

pytestmark = pytest.mark.gpu

SCORE = 2.0 ** -11
INV127 = torch.tensor(1.0) / 127  # fp32


def int8_scale(amax):
    s = amax * INV127
    return torch.where(s > 0, s, torch.ones_like(s))


def want_key(rows):
    """(int8 codes, scale) of a page with these rows [n, 576] (bf16)."""
    mean = (rows.double().sum(0) / rows.shape[0]).float()
    scale = int8_scale(mean.abs().max())
    return torch.round(mean / scale).to(torch.int8), scale


class Case:
    def __init__(self, lengths, h_q=16, s_q=1, seed=0, spare=3, d_v=512):
        g = torch.Generator().manual_seed(seed)
        self.lengths, self.h_q, self.s_q, self.d_v = lengths, h_q, s_q, d_v
        pages = [-(-n // 64) for n in lengths]
        self.blocks = sum(pages) + spare
        perm = torch.randperm(self.blocks, generator=g).to(torch.int32)
        # rows of a page share a direction, as neighbouring tokens do
        self.cache = (torch.randn((self.blocks, 64, 1, 576), generator=g) +
                      torch.randn((self.blocks, 1, 1, 576), generator=g)).to(torch.bfloat16)
        self.q = torch.randn((len(lengths), s_q, h_q, 576), generator=g).to(torch.bfloat16)
        self.table = torch.full((len(lengths), max(1, max(pages))), -1, dtype=torch.int32)
        at = 0
        for b, n in enumerate(pages):
            self.table[b, :n] = perm[at:at + n]
            at += n
        self.keys = torch.zeros((self.blocks, 576), dtype=torch.int8)
        self.scales = torch.ones(self.blocks)
        for b, n in enumerate(lengths):
            for p in range(pages[b]):
                blk = int(self.table[b, p])
                self.keys[blk], self.scales[blk] = want_key(
                    self.cache[blk, :min(64, n - 64 * p), 0])
        self.scale = 1 / math.sqrt(576)

    def sl(self):
        return torch.tensor(self.lengths, dtype=torch.int32, device="cuda")

    def run(self, topk, causal=True, **kw):
        return B.mla_page_sparse_decode(
            self.q.cuda(), self.cache.cuda(), self.keys.cuda(), self.scales.cuda(),
            self.table.cuda(), self.sl(), topk, causal=causal, softmax_scale=self.scale,
            d_v=self.d_v, **kw)

    def seen(self, b, i, causal):
        n = min(self.lengths[b], 64 * self.table.shape[1])
        return max(0, n - self.s_q + 1 + i if causal else n)

    def select(self, b, i, topk, causal=True):
        seen = self.seen(b, i, causal)
        last = -(-seen // 64) - 1
        if last < topk:
            return list(range(last + 1))
        q = self.q[b, i].float()
        unit = int8_scale(q.abs().amax(1))
        code = torch.round(q / unit[:, None])
        blk = self.table[b, :last].long().clamp(0)
        # whole numbers: exact in fp64
        dot = (code.double() @ self.keys[blk].double().T).float()
        score = (dot * unit[:, None]).amax(0) * self.scales[blk]
        order = torch.sort(score, descending=True, stable=True)[1][:topk - 1].tolist()
        return sorted(order) + [last]

    def check(self, got, topk, causal=True):
        torch.cuda.synchronize()
        assert B.device_status() == 0
        out, lse, pages = [t.cpu() for t in got]
        for b in range(len(self.lengths)):
            for i in range(self.s_q):
                seen = self.seen(b, i, causal)
                want = self.select(b, i, topk, causal)
                assert pages[b, i].tolist() == want + [-1] * (topk - len(want)), (b, i)
                if not want:
                    assert (out[b, i] == 0).all() and torch.isneginf(lse[b, i]).all()
                    continue
                t = torch.cat([torch.arange(64 * p, min(64 * p + 64, seen)) for p in want])
                k = self.cache.view(-1, 576)[self.table[b].long()[t // 64] * 64 + t % 64].double()
                x = self.q[b, i].double() @ k.T * self.scale
                want_l = torch.logsumexp(x, 1)
                p = torch.exp(x - want_l[:, None])
                v = k[:, :self.d_v]
                o, size = p @ v, p @ v.abs()
                bound = 2.0 ** -8 * (1 + 2.0 ** -4) * (size + o.abs()) + SCORE * size + 1e-30
                err = (out[b, i].double() - o).abs()
                assert (err <= bound).all(), (b, i, float((err / bound).max()))
                assert ((lse[b, i].double() - want_l).abs() <=
                        SCORE + 2.0 ** -20 * want_l.abs()).all()


# ------------------------------------------------------------------ page keys

def update(c, keys, scales, lengths=None, tail=None, cache=None):
    sl = torch.tensor(c.lengths if lengths is None else lengths, dtype=torch.int32, device="cuda")
    cache = c.cache.cuda() if cache is None else cache
    B.mla_page_keys_update(cache, c.table.cuda(), sl, keys, scales, tail_pages=tail)
    torch.cuda.synchronize()


@pytest.mark.parametrize("lengths", [[1], [63], [64], [65], [0, 200, 0, 1, 129], [1000, 777]])
def test_keys_of_all_pages(lengths):
    c = Case(lengths, seed=len(lengths))
    keys = torch.full((c.blocks, 576), 99, dtype=torch.int8, device="cuda")
    scales = torch.full((c.blocks,), -3.0, device="cuda")
    update(c, keys, scales)
    assert B.device_status() == 0
    owned = torch.zeros(c.blocks, dtype=torch.bool)
    owned[c.table[c.table >= 0].long()] = True
    assert torch.equal(keys.cpu()[owned], c.keys[owned])
    assert torch.equal(scales.cpu()[owned], c.scales[owned])
    # entries of other blocks stay
    assert (keys.cpu()[~owned] == 99).all() and (scales.cpu()[~owned] == -3.0).all()


@pytest.mark.parametrize("tail", [1, 2, 3, 7, 100])
def test_only_the_tail_is_written(tail):
    c = Case([300, 0, 64, 65, 129], seed=tail)
    keys = torch.full((c.blocks, 576), 99, dtype=torch.int8, device="cuda")
    scales = torch.full((c.blocks,), -3.0, device="cuda")
    update(c, keys, scales, tail=tail)
    written = torch.zeros(c.blocks, dtype=torch.bool)
    for b, n in enumerate(c.lengths):
        total = -(-n // 64)
        written[c.table[b, max(0, total - tail):total].long()] = True
    assert torch.equal(keys.cpu()[written], c.keys[written])
    assert torch.equal(scales.cpu()[written], c.scales[written])
    assert (keys.cpu()[~written] == 99).all() and (scales.cpu()[~written] == -3.0).all()


def test_key_values_at_the_edges():
    c = Case([64 * 6 + 10], seed=3, spare=0)
    rows = c.cache[c.table[0].long(), :, 0]  # a copy
    rows[0] = 0                                   # zero page: scale 1, codes 0
    rows[1] = torch.where(torch.arange(64)[:, None] % 2 == 0, 1.0, -1.0)  # cancels to zero
    rows[2] = 2.0 ** -120                         # tiny
    rows[3] = 3.0e38                              # the sum passes the fp32 range
    rows[4, :, :288] = 127.0                      # codes on and between whole numbers
    rows[4, :, 288:] = 0.5
    rows[5] = 2.0 ** -133                         # the scale underflows to a denormal or 0
    rows[6, 10:] = float("nan")                   # rows behind the sequence are not read
    c.cache[c.table[0].long(), :, 0] = rows
    keys = torch.zeros((c.blocks, 576), dtype=torch.int8, device="cuda")
    scales = torch.zeros((c.blocks,), device="cuda")
    update(c, keys, scales)
    for p in range(7):
        blk = int(c.table[0, p])
        code, scale = want_key(c.cache[blk, :min(64, c.lengths[0] - 64 * p), 0])
        assert torch.equal(keys[blk].cpu(), code.clamp(-127, 127)), p
        assert torch.equal(scales[blk].cpu(), scale), p


def test_keys_after_appending_follow_the_new_lengths():
    c = Case([100, 64, 1, 0], seed=4, spare=8)
    c.table = torch.nn.functional.pad(c.table, (0, 1), value=-1)
    spare = [x for x in range(c.blocks) if x not in c.table[c.table >= 0].tolist()]
    c.table[1, 1], c.table[3, 0] = spare[0], spare[1]  # pages that the new tokens need
    keys, scales = c.keys.cuda(), c.scales.cuda()
    c.lengths = [n + 3 for n in c.lengths]
    update(c, keys, scales, tail=2)  # ceil(3 / 64) + 1
    for b, n in enumerate(c.lengths):
        for p in range(-(-n // 64)):
            blk = int(c.table[b, p])
            code, scale = want_key(c.cache[blk, :min(64, n - 64 * p), 0])
            assert torch.equal(keys[blk].cpu(), code) and torch.equal(scales[blk].cpu(), scale)


def test_key_update_reports_bad_inputs_and_stays_in_bounds():
    c = Case([70, 130], seed=5)
    keys, scales = torch.zeros_like(c.keys).cuda(), torch.zeros_like(c.scales).cuda()
    update(c, keys, scales, lengths=[1000, 130])  # cut to the table's three pages
    assert B.device_status() >> 16 == B.MLA_DEVERR_BAD_INDEX
    for p in range(3):
        blk = int(c.table[1, p])
        code, scale = want_key(c.cache[blk, :min(64, 130 - 64 * p), 0])
        assert torch.equal(keys[blk].cpu(), code) and torch.equal(scales[blk].cpu(), scale)


def test_key_update_writes_no_key_for_a_bad_block():
    # a bad id must not touch the key of block 0, which another sequence's full page owns
    c = Case([64 * 3, 64 * 2 + 5], seed=6)
    c.table[c.table == 0] = int(c.table[0, 0])
    c.table[0, 0] = 0
    for b, n in enumerate(c.lengths):
        for p in range(-(-n // 64)):
            blk = int(c.table[b, p])
            c.keys[blk], c.scales[blk] = want_key(c.cache[blk, :min(64, n - 64 * p), 0])
    named = torch.zeros(c.blocks, dtype=torch.bool)
    for bad in (-1, c.blocks, -2 ** 31, 2 ** 31 - 1):
        c.table[1, 2] = bad  # the page of five rows
        keys = torch.full((c.blocks, 576), 99, dtype=torch.int8, device="cuda")
        scales = torch.full((c.blocks,), -3.0, device="cuda")
        update(c, keys, scales)
        assert B.device_status() >> 16 == B.MLA_DEVERR_BAD_INDEX
        named[:] = False
        named[torch.cat([c.table[0], c.table[1, :2]]).long()] = True
        assert torch.equal(keys.cpu()[named], c.keys[named])
        assert torch.equal(scales.cpu()[named], c.scales[named])
        assert (keys.cpu()[~named] == 99).all() and (scales.cpu()[~named] == -3.0).all()
        update(c, keys, scales, tail=1)
        assert B.device_status() >> 16 == B.MLA_DEVERR_BAD_INDEX
        assert torch.equal(keys.cpu()[0], c.keys[0]) and torch.equal(scales.cpu()[0], c.scales[0])


# ------------------------------------------------------------------ page-selected decode

@pytest.mark.parametrize("h_q", [1, 5, 16, 31, 33, 64, 65, 128, 130])
def test_heads(h_q):
    c = Case([900, 1500, 64], h_q=h_q, seed=h_q)
    c.check(c.run(5), 5)


@pytest.mark.parametrize("topk", [1, 2, 3, 8, 15, 16, 17, 40])
def test_topk(topk):
    c = Case([1024, 961, 1000, 63, 0, 1], seed=topk)
    c.check(c.run(topk), topk)


@pytest.mark.parametrize("lengths", [[0], [1], [64], [65], [128], [129], [0, 0, 193],
                                     [320, 321, 319]])
def test_lengths(lengths):
    c = Case(lengths, seed=len(lengths))
    c.check(c.run(2), 2)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("s_q", [2, 3, 70])
def test_several_query_tokens(s_q, causal):
    # sequences shorter than s_q: the first queries see nothing; 64 and 65 end
    # different pages for neighbouring queries
    c = Case([1, 2, 65, 130, 700, 0], s_q=s_q, h_q=8, seed=s_q)
    c.check(c.run(3, causal=causal), 3, causal)


def test_many_pages_and_chunks():
    # several score CTAs (128 pages each), select passes over more than 256 pages
    c = Case([64 * 700 + 3, 64 * 128, 64 * 129, 64 * 257 + 1], seed=7)
    for topk in (1, 31, 300):
        c.check(c.run(topk), topk)


@pytest.mark.parametrize("h_q", [16, 200])
@pytest.mark.parametrize("pages", [512, 513, 4096, 4097, 6001])
def test_long_tables(pages, h_q):
    # pages of few blocks: many equal scores, and tables beyond one chunk of the selection
    c = Case([64 * 300], h_q=h_q, seed=pages)
    g = torch.Generator().manual_seed(pages)
    c.lengths = [64 * pages + 5]
    c.table = torch.randint(0, 300, (1, pages + 1), generator=g).to(torch.int32)
    for topk in (2, 33, 500):
        c.check(c.run(topk), topk)


@pytest.mark.parametrize("n,h_q,pages,topk", [(40, 128, 130, 128), (40, 128, 40, 16),
                                              (76, 64, 130, 120), (76, 64, 20, 8),
                                              (5, 16, 130, 128), (100, 16, 70, 64)])
def test_plans_with_and_without_whole_parts_per_query(n, h_q, pages, topk):
    # sequences that share the pages of one cache
    c = Case([64 * pages], h_q=h_q, seed=28)
    g = torch.Generator().manual_seed(28)
    c.lengths = torch.randint(64 * topk, 64 * pages + 1, (n,), generator=g).tolist()
    c.table = torch.stack([c.table[0][torch.randperm(pages, generator=g)] for _ in range(n)])
    c.q = torch.randn((n, 1, h_q, 576), generator=g).to(torch.bfloat16)
    c.check(c.run(topk), topk)


def test_d_v_576():
    c = Case([700, 100], seed=8, d_v=576)
    c.check(c.run(4), 4)


def test_ties_take_the_lowest_pages():
    c = Case([64 * 20], seed=9)
    c.keys[:] = c.keys[0]
    c.scales[:] = c.scales[0]
    pages = c.run(6)[2]
    assert pages.cpu().tolist() == [[[0, 1, 2, 3, 4, 19]]]
    c.check(c.run(6), 6)
    # scores of both signs of zero, and a border inside equal scores
    c.keys[:] = 0
    c.keys[c.table[0, 7].long()] = 1
    c.q[..., :] = c.q.abs()
    assert c.run(3)[2].cpu().tolist() == [[[0, 7, 19]]]
    c.q[..., :] = -c.q
    assert c.run(3)[2].cpu().tolist() == [[[0, 1, 19]]]
    c.check(c.run(3), 3)


def test_zero_query_and_equal_products():
    c = Case([64 * 12 + 5], seed=10)
    c.q[:] = 0
    c.check(c.run(4), 4)
    assert c.run(4)[2].cpu().tolist() == [[[0, 1, 2, 12]]]


@pytest.mark.parametrize("h_q", [1, 130])
def test_scores_that_underflow_tie_with_zero(h_q):
    # negative products that underflow on the even pages, exact zeros on the odd ones
    c = Case([64 * 12], h_q=h_q, seed=26)
    c.q[:] = 2.0 ** -100
    c.keys[:] = 0
    c.keys[c.table[0, 0:12:2].long()] = -1
    c.scales[:] = 2.0 ** -90
    assert c.run(5)[2].cpu().tolist() == [[[0, 1, 2, 3, 11]]]
    c.check(c.run(5), 5)


def test_negative_scores_are_ordered():
    c = Case([64 * 40], h_q=1, seed=11)
    base = torch.randint(1, 127, (576,), dtype=torch.int8)
    for p in range(40):  # every score negative, descending with the page
        c.keys[c.table[0, p].long()] = -base
        c.scales[c.table[0, p].long()] = 1.0 + p
    c.q[:] = base.to(torch.bfloat16)
    assert c.run(4)[2].cpu().tolist() == [[[0, 1, 2, 39]]]
    c.check(c.run(4), 4)


@pytest.mark.parametrize("kind", ["halves", "random", "tiny", "huge"])
def test_query_codes(kind):
    """One head against one-hot keys: the score of page p is the code of dim p, so the order of
    the pages shows the codes."""
    c = Case([64 * 577], h_q=1, seed=21, spare=0)
    c.keys[c.table[0, :576].long()] = torch.diag(torch.full((576,), 127)).to(torch.int8)
    c.scales[:] = 1.0
    g = torch.Generator().manual_seed(22)
    if kind == "halves":  # scale 1: whole numbers and halves, where ties go to the even code
        x = torch.arange(576) / 2.0 - 100
        x[0] = 127.0
        x = x.clamp(-127, 127)
    else:
        x = torch.randn(576, generator=g)
        # below and above the range where the reciprocal of the scale is used
        x = x * {"random": 1.0, "tiny": 2.0 ** -105, "huge": 2.0 ** 110}[kind]
    c.q[0, 0, 0] = x.to(torch.bfloat16)
    c.cache[:] = 0
    q = c.q.cuda()
    for topk in (2, 17, 100, 288, 400, 575):
        pages = B.mla_page_sparse_decode(q, c.cache.cuda(), c.keys.cuda(), c.scales.cuda(),
                                         c.table.cuda(), c.sl(), topk)[2]
        assert pages[0, 0].tolist() == c.select(0, 0, topk)
    assert B.device_status() == 0


def test_all_pages_taken_is_the_dense_decode():
    c = Case([700, 90, 0], h_q=32, s_q=2, seed=12)
    out, lse, _ = c.run(c.table.shape[1])
    meta, ns, parts = B.mla_get_metadata(c.sl(), 64, 1)
    o2, l2 = B.mla_decode_fwd(c.q.cuda(), c.cache.cuda(), c.table.cuda(), c.sl(), 512, meta, ns,
                              parts, causal=True, softmax_scale=c.scale)
    c.check((out, lse, c.run(c.table.shape[1])[2]), c.table.shape[1])
    assert ((out.float() - o2.float()).abs() <= 2.0 ** -6 * (1 + o2.float().abs())).all()
    fin = torch.isfinite(l2)
    assert torch.equal(torch.isfinite(lse), fin) and ((lse - l2)[fin].abs() <= 2 * SCORE).all()


def test_repeats_give_the_same_bits():
    c = Case([64 * 200 + 9, 3000], h_q=128, seed=13)
    a = c.run(9)
    for _ in range(3):
        assert all(torch.equal(x, y) for x, y in zip(a, c.run(9)))


def test_stream_and_graph_with_new_lengths():
    c = Case([1000, 640, 70], seed=14)
    q, cache, table, sl = c.q.cuda(), c.cache.cuda(), c.table.cuda(), c.sl()
    keys, scales = torch.zeros_like(c.keys).cuda(), torch.ones_like(c.scales).cuda()
    out = torch.empty((3, 1, 16, 512), dtype=torch.bfloat16, device="cuda")
    lse = torch.empty((3, 1, 16), device="cuda")
    pages = torch.empty((3, 1, 4), dtype=torch.int32, device="cuda")
    ws = torch.empty(B.mla_page_sparse_workspace_size(3, 1, 16, 512, table.shape[1], 4, 100),
                     dtype=torch.uint8, device="cuda")

    def step():
        B.mla_page_keys_update(cache, table, sl, keys, scales)
        B.mla_page_sparse_decode(q, cache, keys, scales, table, sl, 4, softmax_scale=c.scale,
                                 num_sm_parts=100, pages=pages, out=out, lse=lse, workspace=ws)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    side.synchronize()
    c.check((out, lse, pages), 4)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    c.lengths = [777, 1, 64]
    sl.copy_(c.sl())
    for b, n in enumerate(c.lengths):
        for p in range(-(-n // 64)):
            blk = int(c.table[b, p])
            c.keys[blk], c.scales[blk] = want_key(c.cache[blk, :min(64, n - 64 * p), 0])
    c.q = c.q.flip(3).contiguous()
    q.copy_(c.q)
    graph.replay()
    c.check((out, lse, pages), 4)


def test_bad_blocks_and_lengths():
    c = Case([500, 450], seed=15)
    good = c.table.clone()
    c.table[0, 2] = c.blocks + 9
    got = c.run(8)  # every page: block 0 stands in for the bad one
    assert B.device_status() >> 16 == B.MLA_DEVERR_BAD_INDEX
    c.table[0, 2] = 0
    c.check(got, 8)
    c.table = good
    c.lengths = [100000, 450]  # cut to the table's eight pages
    got = c.run(3)
    assert B.device_status() >> 16 == B.MLA_DEVERR_BAD_INDEX
    c.check(got, 3)


def test_slot_trace_names_the_taken_rows():
    c = Case([64 * 9 + 3, 200], seed=16)
    width = c.table.shape[1]
    trace = torch.full((2 * 2 * width * 64,), -9, dtype=torch.int32, device="cuda")
    B.mla_set_slot_trace(trace)
    try:
        got = c.run(3)
        torch.cuda.synchronize()
    finally:
        B.mla_set_slot_trace(None)
    plane = 2 * 3 * 64
    want = torch.full((plane,), -9, dtype=torch.int32)
    for b in range(2):
        for j, p in enumerate(c.select(b, 0, 3)):
            at = (b * 3 + j) * 64
            want[at:at + 64] = c.table[b, p] * 64 + torch.arange(64, dtype=torch.int32)
    assert torch.equal(trace[:plane].cpu(), want)
    assert torch.equal(trace[plane:2 * plane].cpu(), want)
    c.check(got, 3)


def test_wider_indexes_and_strided_inputs():
    c = Case([900, 333], h_q=16, s_q=2, seed=19)
    want = c.run(4)
    q = torch.empty((2, 2, 16, 600), dtype=torch.bfloat16, device="cuda")[..., :576]
    q.copy_(c.q)
    table = torch.empty((2, 2 * c.table.shape[1]), dtype=torch.int64, device="cuda")[:, ::2]
    table.copy_(c.table)
    keys, scales = c.keys.cuda(), c.scales.cuda()
    got = B.mla_page_sparse_decode(q, c.cache.cuda(), keys, scales, table, c.sl().long(), 4,
                                   softmax_scale=c.scale)
    assert all(torch.equal(x, y) for x, y in zip(got, want))
    B.mla_page_keys_update(c.cache.cuda(), table, c.sl().long(), keys, scales)
    owned = c.table[c.table >= 0].long()
    assert torch.equal(keys.cpu()[owned], c.keys[owned])


def test_an_empty_batch():
    c = Case([500], seed=27)
    none = c.table[:0].cuda()
    got = B.mla_page_sparse_decode(c.q[:0].cuda(), c.cache.cuda(), c.keys.cuda(), c.scales.cuda(),
                                   none, c.sl()[:0], 3)
    assert [tuple(t.shape) for t in got] == [(0, 1, 16, 512), (0, 1, 16), (0, 1, 3)]
    B.mla_page_keys_update(c.cache.cuda(), none, c.sl()[:0], c.keys.cuda(), c.scales.cuda())


def test_int64_blocks_and_lengths_past_int32_are_out_of_range():
    c = Case([500, 450], seed=20)
    keys, scales = c.keys.cuda(), c.scales.cuda()
    args = (c.q.cuda(), c.cache.cuda(), keys, scales)
    table, sl = c.table.long(), c.sl().long()
    table[0, 2] += 2 ** 32
    got = B.mla_page_sparse_decode(*args, table.cuda(), sl, 8, softmax_scale=c.scale)
    assert B.device_status() >> 16 == B.MLA_DEVERR_BAD_INDEX
    good, c.table[0, 2] = int(c.table[0, 2]), 0  # block 0 stands in for it
    c.check(got, 8)
    # its key is not written
    keys[:] = 99
    B.mla_page_keys_update(c.cache.cuda(), table.cuda(), sl, keys, scales)
    assert B.device_status() >> 16 == B.MLA_DEVERR_BAD_INDEX
    assert (keys[good] == 99).all()
    # a length of 2^32 + 450 is past the table, not 450
    c.table[0, 2] = good
    sl[1] += 2 ** 32
    got = B.mla_page_sparse_decode(*args[:2], c.keys.cuda(), c.scales.cuda(), c.table.cuda(), sl, 3,
                                   softmax_scale=c.scale)
    assert B.device_status() >> 16 == B.MLA_DEVERR_BAD_INDEX
    c.lengths = [500, 512]
    c.check(got, 3)


def test_two_streams_at_once():
    a, b = Case([64 * 150 + 3] * 3, h_q=128, seed=23), Case([5000, 64], h_q=16, seed=24)
    ta = (a.q.cuda(), a.cache.cuda(), a.keys.cuda(), a.scales.cuda(), a.table.cuda(), a.sl())
    tb = (b.q.cuda(), b.cache.cuda(), b.keys.cuda(), b.scales.cuda(), b.table.cuda(), b.sl())
    sa, sb = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    got = []
    for _ in range(8):
        with torch.cuda.stream(sa):
            x = B.mla_page_sparse_decode(*ta, 7, softmax_scale=a.scale)
        with torch.cuda.stream(sb):
            y = B.mla_page_sparse_decode(*tb, 3, softmax_scale=b.scale)
        got.append((x, y))
    for x, y in got:
        a.check(x, 7)
        b.check(y, 3)


def test_rejects_wrong_arguments():
    c = Case([500, 450], seed=17)
    good = dict(q=c.q.cuda(), kcache=c.cache.cuda(), page_keys=c.keys.cuda(),
                page_scales=c.scales.cuda(), block_table=c.table.cuda(), cache_seqlens=c.sl(),
                topk_pages=3)
    for change in [dict(q=c.q), dict(q=good["q"].float()), dict(q=good["q"][..., :512]),
                   dict(kcache=c.cache), dict(kcache=good["kcache"].view(-1, 576)),
                   dict(page_keys=c.keys), dict(page_keys=good["page_keys"].float()),
                   dict(page_keys=good["page_keys"][:2]), dict(page_scales=c.scales),
                   dict(page_scales=good["page_scales"][:2]), dict(block_table=c.table),
                   dict(block_table=good["block_table"][:1]),
                   dict(cache_seqlens=good["cache_seqlens"].float()), dict(topk_pages=0),
                   dict(softmax_scale=0.0), dict(d_v=500),
                   dict(workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))]:
        with pytest.raises((ValueError, B.MLAError)):
            B.mla_page_sparse_decode(**(good | change))
    keys = {k: good[k] for k in ("kcache", "block_table", "cache_seqlens", "page_keys",
                                 "page_scales")}
    for change in [dict(kcache=c.cache), dict(page_keys=good["page_keys"][:, :512]),
                   dict(cache_seqlens=good["cache_seqlens"][:1]), dict(tail_pages=0)]:
        with pytest.raises((ValueError, B.MLAError)):
            B.mla_page_keys_update(**(keys | change))


# ------------------------------------------------------------------ together

def test_a_prompt_and_decode_steps_with_all_of_the_operators():
    """Prompts of two sequences and three decode steps: tokens appended (norm, rotation) to a
    bf16 cache, the page keys kept, and each step decoded over the selected pages."""
    g = torch.Generator().manual_seed(18)
    c = Case([0, 0], h_q=16, seed=18, spare=24)
    lengths = [64 * 7 + 61, 64 * 9]
    perm = torch.randperm(c.blocks, generator=g).to(torch.int32)
    c.table = perm[:22].view(2, 11).contiguous()
    cache = torch.zeros((c.blocks, 64, 1, 576), dtype=torch.bfloat16, device="cuda")
    keys, scales = c.keys.cuda(), c.scales.cuda()
    gain = 1 + 0.1 * torch.randn(512, generator=g)

    def append(first, count):
        pos = torch.cat([torch.arange(f, f + n) for f, n in zip(first, count)])
        slots = torch.cat([c.table[b].long()[torch.arange(f, f + n) // 64] * 64 +
                           torch.arange(f, f + n) % 64
                           for b, (f, n) in enumerate(zip(first, count))])
        kv = torch.randn((len(pos), 576), generator=g).to(torch.bfloat16).cuda()
        B.mla_cache_append(kv, slots.to(torch.int32).cuda(), cache,
                           positions=pos.to(torch.int32).cuda(), norm_gain=gain.cuda())

    append([0, 0], lengths)
    c.lengths = lengths
    B.mla_page_keys_update(cache, c.table.cuda(), c.sl(), keys, scales)
    for _ in range(5):  # the first sequence crosses into a new page on the way
        append(c.lengths, [1, 1])
        c.lengths = [n + 1 for n in c.lengths]
        B.mla_page_keys_update(cache, c.table.cuda(), c.sl(), keys, scales, tail_pages=1)
        c.q = torch.randn((2, 1, 16, 576), generator=g).to(torch.bfloat16)
        got = B.mla_page_sparse_decode(c.q.cuda(), cache, keys, scales, c.table.cuda(), c.sl(), 4,
                                       softmax_scale=c.scale)
        torch.cuda.synchronize()
        c.cache, c.keys, c.scales = cache.cpu(), keys.cpu(), scales.cpu()
        for b, n in enumerate(c.lengths):
            for p in range(-(-n // 64)):
                blk = int(c.table[b, p])
                code, scale = want_key(c.cache[blk, :min(64, n - 64 * p), 0])
                assert torch.equal(c.keys[blk], code) and torch.equal(c.scales[blk], scale)
        c.check(got, 4)

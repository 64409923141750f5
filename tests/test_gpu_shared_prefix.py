"""mla_shared_prefix_decode_fwd against attention over the joined sequence in
fp64.

Tolerances.  The probabilities enter the second product as bf16 (half a step:
2^-8 of each), and the output is rounded to bf16 (2^-8 of it), so |o - o64| <=
2^-8 (A + |o64|) with A = sum_i p_i |v_i|.  The scores are fp32 sums of 576
exact products: an error of at most 576 * 2^-24 * sum |q_j k_j| * scale, under
2^-9 at the sizes here and in practice far below; it moves every p by that
relative amount and the LSE by that much.  SCORE bounds it by 2^-11 (sums of
independent roundings: sqrt(576) * 2^-24 * 40 < 2^-13).
"""
import math

import pytest
import torch

import oracle
from mla_paged_kv_03_b200 import binding as B
from parity_util import assert_lse_close, assert_out_close

pytestmark = pytest.mark.gpu

SCORE = 2.0 ** -11


class Case:
    def __init__(self, lengths, prefix_len, s_q, h_q, seed=0, spare=3, std=1.0, device="cuda"):
        g = torch.Generator().manual_seed(seed)
        self.lengths, self.prefix_len, self.s_q, self.h_q = lengths, prefix_len, s_q, h_q
        pages = [-(-n // 64) for n in [prefix_len] + lengths]
        self.blocks = sum(pages) + spare
        perm = torch.randperm(self.blocks, generator=g).to(torch.int32)
        self.cache = torch.randn((self.blocks, 64, 1, 576), generator=g).to(torch.bfloat16)
        self.q = (std * torch.randn((len(lengths), s_q, h_q, 576), generator=g)).to(torch.bfloat16)
        self.prefix_table = perm[:pages[0]].clone()
        width = max(1, max(pages[1:]))
        self.table = torch.full((len(lengths), width), -1, dtype=torch.int32)
        at = pages[0]
        for b, n in enumerate(pages[1:]):
            self.table[b, :n] = perm[at:at + n]
            at += n
        self.scale = 1 / math.sqrt(576)
        self.device = torch.device(device)

    def dev(self):
        d = self.device
        return (self.q.to(d), self.cache.to(d), self.prefix_table.to(d), self.table.to(d),
                torch.tensor(self.lengths, dtype=torch.int32, device=d))

    def run(self, causal=True, parts=None, t=None, **kw):
        q, cache, pt, table, sl = t or self.dev()
        meta, ns, n = B.mla_shared_prefix_get_metadata(sl, self.prefix_len, self.s_q * self.h_q,
                                                       num_sm_parts=parts)
        return B.mla_shared_prefix_decode_fwd(q, cache, pt, self.prefix_len, table, sl, meta, ns,
                                              n, causal=causal, softmax_scale=self.scale, **kw)

    def rows_of(self, blocks, n):
        t = torch.arange(n)
        return self.cache.view(-1, 576)[blocks.long()[t // 64] * 64 + t % 64].double()

    def check(self, got, causal=True, seqs=None, score=SCORE):
        torch.cuda.synchronize()
        assert B.device_status() == 0
        out, lse = got[0].cpu().double(), got[1].cpu().double()
        head = self.rows_of(self.prefix_table, self.prefix_len)
        for b in seqs if seqs is not None else range(len(self.lengths)):
            n = self.lengths[b]
            k = torch.cat([head, self.rows_of(self.table[b], n)]).to(self.device)
            for i in range(self.s_q):
                seen = len(k) - self.s_q + 1 + i if causal else len(k)
                ko = k[:max(seen, 0)]
                o, l = out[b, i].to(self.device), lse[b, i].to(self.device)
                if len(ko) == 0:
                    assert (o == 0).all() and torch.isneginf(l).all()
                    continue
                x = self.q[b, i].to(self.device).double() @ ko.T * self.scale
                want_l = torch.logsumexp(x, 1)
                p = torch.exp(x - want_l[:, None])
                want, size = p @ ko[:, :512], p @ ko[:, :512].abs()
                bound = 2.0 ** -8 * (1 + 2.0 ** -4) * (size + want.abs()) + score * size + 1e-30
                err = (o - want).abs()
                assert (err <= bound).all(), (b, i, float((err / bound).max()))
                assert ((l - want_l).abs() <= score + 2.0 ** -20 * want_l.abs()).all()


@pytest.mark.parametrize("h_q", [1, 5, 16, 20, 64, 96, 128])
def test_heads(h_q):
    c = Case([40, 130, 1], 200, 1, h_q, seed=h_q)
    c.check(c.run())


@pytest.mark.parametrize("prefix_len", [1, 63, 64, 65, 127, 128, 129, 255, 256, 257, 700])
def test_prefix_lengths(prefix_len):
    c = Case([30, 64, 65, 300], prefix_len, 1, 16, seed=prefix_len)
    c.check(c.run())


@pytest.mark.parametrize("lengths", [[0], [1], [0, 0, 0], [0, 5, 0, 257], [128], [513, 1, 64]])
def test_own_lengths(lengths):
    c = Case(lengths, 300, 1, 32, seed=len(lengths))
    c.check(c.run())


@pytest.mark.parametrize("lengths", [[0, 3], [400, 64]])
def test_no_prefix_is_a_plain_decode(lengths):
    c = Case(lengths, 0, 1, 16, seed=8)
    c.check(c.run())
    c.check(c.run(causal=False), causal=False)


@pytest.mark.parametrize("s_q", [2, 3, 9])
@pytest.mark.parametrize("prefix_len", [0, 1, 4, 130])
def test_several_query_tokens(s_q, prefix_len):
    # own parts shorter than s_q: the first queries see less than the prefix, or nothing
    c = Case([0, 1, 2, 5, 70, 200], prefix_len, s_q, 16, seed=s_q)
    c.check(c.run())
    c.check(c.run(causal=False), causal=False)


def test_more_rows_than_a_group_per_sequence():
    c = Case([65, 300], 260, 3, 128, seed=1)  # 384 rows: three groups
    c.check(c.run())
    c = Case([65, 300, 2], 260, 3, 50, seed=2)  # 150 rows: groups of 128 and 22
    c.check(c.run())


@pytest.mark.parametrize("parts", [1, 2, 7, 74, 200])
def test_split_counts(parts):
    c = Case([90, 700, 0, 33], 1500, 1, 24, seed=parts)
    c.check(c.run(parts=parts))


def test_growing_scores_rescale():
    # keys whose scores grow along the prefix and into the own tokens
    c = Case([300, 300], 900, 1, 16, seed=5)
    ramp = torch.linspace(0.1, 4.0, c.blocks * 64)
    order = torch.cat([c.prefix_table, c.table[0], c.table[1]]).long()
    for i, blk in enumerate(order.tolist()):
        c.cache[blk] = (c.q[0, 0, 0].float() * ramp[i * 64:(i + 1) * 64].view(64, 1, 1) * 0.3 +
                        0.2 * c.cache[blk].float()).to(torch.bfloat16)
    # the scores reach about 60: the bound on their error scales with them
    c.check(c.run(), score=2.0 ** -8)


def test_large_batch_and_long_prefix():
    c = Case([(37 * i) % 400 for i in range(70)], 9000, 1, 16, seed=6)
    c.check(c.run(), seqs=[0, 1, 33, 69])
    c = Case([5 * i for i in range(20)], 4097, 1, 128, seed=7)
    c.check(c.run(), seqs=[0, 7, 19])


def test_equals_the_decode_over_the_joined_sequence():
    c = Case([10, 200, 64], 640, 2, 32, seed=9)
    out, lse = c.run()
    joined = torch.cat([c.prefix_table.expand(3, -1), c.table], 1)
    sl = torch.tensor([640 + n for n in c.lengths], dtype=torch.int32)
    ro, rl = oracle.dense_decode(c.q, c.cache, joined, sl, 512, c.scale, causal=True)
    assert_out_close(out, ro)
    assert_lse_close(lse, rl)


def test_reused_and_misaligned_buffers():
    # outputs and a workspace on 16- but not 32-byte boundaries give the same bits
    c = Case([10, 200, 64], 640, 1, 16, seed=10)
    t = c.dev()
    out, lse = c.run(t=t)
    n = B.mla_shared_prefix_workspace_size(3, 16, 640, 74)
    raw = torch.full((n + 64,), 255, dtype=torch.uint8, device="cuda")
    o = torch.empty(out.numel() + 8, dtype=torch.bfloat16, device="cuda")[8:].view(out.shape)
    for _ in range(2):
        o2, l2 = c.run(t=t, out=o, workspace=raw[16:16 + n], parts=74)
        assert torch.equal(o2, out) and torch.equal(l2, lse)


def test_stream_and_graph():
    c = Case([10, 200, 64], 640, 1, 16, seed=11)
    q, cache, pt, table, sl = c.dev()
    out, lse = torch.empty((3, 1, 16, 512), dtype=torch.bfloat16, device="cuda"), \
        torch.empty((3, 1, 16), device="cuda")
    ws = torch.empty(B.mla_shared_prefix_workspace_size(3, 16, 640, 74), dtype=torch.uint8,
                     device="cuda")

    def step():
        c.run(t=(q, cache, pt, table, sl), out=out, lse=lse, workspace=ws, parts=74)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    side.synchronize()
    want = out.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    out.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    # new lengths and queries in the same buffers: the plan is part of the graph
    c.lengths = [64, 1, 3]
    sl.copy_(torch.tensor(c.lengths, dtype=torch.int32))
    c.q = c.q.flip(2).contiguous()
    q.copy_(c.q)
    graph.replay()
    c.check((out, lse))


def test_bad_blocks_and_lengths_follow_the_dense_reading():
    # an out-of-range block reads block 0; a length past the table is cut; both are recorded
    c = Case([70, 64], 130, 1, 16, seed=12)
    t = list(c.dev())
    t[2] = t[2].clone()
    t[2][1] = c.blocks + 7
    c.prefix_table[1] = 0
    got = c.run(t=t)
    assert B.device_status() >> 16 == B.MLA_DEVERR_BAD_INDEX
    c.check(got)
    t[2] = c.prefix_table.cuda()
    t[4] = torch.tensor([1000, 64], dtype=torch.int32, device="cuda")
    got = c.run(t=t)
    assert B.device_status() >> 16 == B.MLA_DEVERR_BAD_INDEX
    c.lengths = [128, 64]
    c.table[0, 1] = c.table[0, 1] if c.table[0, 1] >= 0 else 0
    c.check(got)


def test_a_plan_of_other_units_is_refused_on_the_device():
    c = Case([70, 64], 130, 1, 16, seed=13)
    q, cache, pt, table, sl = c.dev()
    meta, ns, n = B.mla_shared_prefix_get_metadata(sl, 0, 16)  # without the prefix
    out = torch.full((2, 1, 16, 512), 3.0, dtype=torch.bfloat16, device="cuda")
    B.mla_shared_prefix_decode_fwd(q, cache, pt, 130, table, sl, meta, ns, n, out=out)
    assert B.device_status() >> 16 == B.MLA_DEVERR_BAD_INDEX
    assert (out == 3.0).all()
    c.check(c.run())


def test_a_plan_of_another_prefix_length_is_refused_on_the_device():
    c = Case([70, 64], 130, 1, 16, seed=13)
    q, cache, pt, table, sl = c.dev()
    meta, ns, n = B.mla_shared_prefix_get_metadata(sl, 64, 16)
    out = torch.full((2, 1, 16, 512), 3.0, dtype=torch.bfloat16, device="cuda")
    B.mla_shared_prefix_decode_fwd(q, cache, pt, 130, table, sl, meta, ns, n, out=out)
    assert B.device_status() >> 16 == B.MLA_DEVERR_BAD_INDEX
    assert (out == 3.0).all()
    c.check(c.run())


def assert_refused(c, plan):
    q, cache, pt, table, sl = c.dev()
    out = torch.full((*c.q.shape[:3], 512), 3.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full(c.q.shape[:3], 3.0, device="cuda")
    B.mla_shared_prefix_decode_fwd(q, cache, pt, c.prefix_len, table, sl, *plan, out=out, lse=lse)
    assert B.device_status() >> 16 == B.MLA_DEVERR_BAD_INDEX
    assert (out == 3.0).all() and (lse == 3.0).all()
    c.check(c.run())


@pytest.mark.parametrize("prefix_len", [0, 130])
def test_a_plan_of_other_rows_with_as_many_units_is_refused(prefix_len):
    # 2 x 256 rows and 4 x 128 rows: as many units over the prefix, and as many own ones
    c = Case([70, 64, 300, 0], prefix_len, 1, 128, seed=14)
    two = torch.tensor([70, 64], dtype=torch.int32, device="cuda")
    assert_refused(c, B.mla_shared_prefix_get_metadata(two, prefix_len, 256))
    c = Case([70, 64], prefix_len, 2, 128, seed=15)
    four = torch.tensor([70, 64, 300, 0], dtype=torch.int32, device="cuda")
    assert_refused(c, B.mla_shared_prefix_get_metadata(four, prefix_len, 128))


@pytest.mark.parametrize("made,used", [(74, 7), (9, 4), (200, 199)])
def test_a_plan_of_other_parts_is_refused(made, used):
    c = Case([700, 64, 1000], 1500, 1, 16, seed=16)
    meta, ns, _ = B.mla_shared_prefix_get_metadata(c.dev()[4], 1500, 16, num_sm_parts=made)
    assert_refused(c, (meta, ns, used))


def test_a_short_num_splits_is_refused():
    # num_splits of a smaller batch beside matching metadata
    c = Case([70, 64, 300], 130, 1, 16, seed=17)
    meta, ns, n = B.mla_shared_prefix_get_metadata(c.dev()[4], 130, 16)
    assert ns.numel() == 1 + 3 + 1
    assert_refused(c, (meta, ns[:-1], n))
    assert_refused(c, (meta, ns[:1].clone(), n))


@pytest.mark.parametrize("prefix_len", [0, 130])
def test_an_empty_batch(prefix_len):
    c = Case([70], prefix_len, 1, 16, seed=18)
    q, cache, pt, table, sl = c.dev()
    plan = B.mla_shared_prefix_get_metadata(sl[:0], prefix_len, 16)
    out, lse = B.mla_shared_prefix_decode_fwd(q[:0], cache, pt, prefix_len, table[:0], sl[:0],
                                              *plan)
    assert out.shape == (0, 1, 16, 512) and lse.shape == (0, 1, 16)


def test_wider_indexes_and_strided_inputs():
    c = Case([70, 64, 0], 200, 2, 16, seed=21)
    want = c.run()
    q, cache, pt, table, sl = c.dev()
    wide = torch.empty((3, 2, 16, 640), dtype=torch.bfloat16, device="cuda")[..., :576]
    wide.copy_(q)
    got = c.run(t=(wide, cache, pt.long(), table.long().t().contiguous().t(), sl))
    assert all(torch.equal(x, y) for x, y in zip(got, want))


def test_rejects_outputs_and_workspaces_of_other_shapes():
    c = Case([70, 64], 130, 1, 16, seed=13)
    for bad in (dict(out=torch.empty((2, 1, 15, 512), dtype=torch.bfloat16, device="cuda")),
                dict(out=torch.empty((2, 1, 16, 512), device="cuda")),
                dict(out=torch.empty((2, 1, 16, 1024), dtype=torch.bfloat16,
                                     device="cuda")[..., ::2]),
                dict(lse=torch.empty((2, 16), device="cuda")),
                dict(lse=torch.empty((2, 1, 16))),
                dict(workspace=torch.empty(1 << 24, dtype=torch.uint8))):
        with pytest.raises(ValueError):
            c.run(**bad)


def test_slot_trace_names_the_rows_read():
    c = Case([70, 200], 130, 1, 16, seed=14)
    width = c.table.shape[1]
    plane = (3 + 2 * width) * 64
    trace = torch.full((2 * plane,), -9, dtype=torch.int32, device="cuda")
    B.mla_set_slot_trace(trace)
    try:
        c.check(c.run())
    finally:
        B.mla_set_slot_trace(None)
    for p in (trace[:plane].cpu(), trace[plane:].cpu()):
        want = torch.full((plane,), -9, dtype=torch.int32)
        tables = [(0, c.prefix_table, 130)] + [(3 + b * width, c.table[b], n)
                                               for b, n in enumerate(c.lengths)]
        for first, table, n in tables:
            for page in range(-(-n // 64)):
                at = (first + page) * 64
                want[at:at + 64] = table[page] * 64 + torch.arange(64, dtype=torch.int32)
        assert torch.equal(p, want)


def test_rejects_wrong_arguments():
    c = Case([70, 64], 130, 1, 16, seed=15)
    q, cache, pt, table, sl = c.dev()
    meta, ns, n = B.mla_shared_prefix_get_metadata(sl, 130, 16)
    good = dict(q=q, kcache=cache, prefix_table=pt, prefix_len=130, block_table=table,
                cache_seqlens=sl, metadata=meta, num_splits=ns, num_sm_parts=n)
    for change in [dict(q=q[..., :512]), dict(q=q.float()), dict(q=q.cpu()),
                   dict(kcache=cache.view(-1, 576)), dict(prefix_table=None),
                   dict(prefix_table=pt[:2]), dict(prefix_len=-1), dict(block_table=table[:1]),
                   dict(cache_seqlens=sl.cpu()), dict(cache_seqlens=sl.float()),
                   dict(metadata=meta[:5]), dict(metadata=meta.cpu()), dict(softmax_scale=0.0),
                   dict(workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))]:
        with pytest.raises((ValueError, B.MLAError)):
            B.mla_shared_prefix_decode_fwd(**(good | change))

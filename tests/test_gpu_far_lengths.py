"""Lengths that no cache holds (uninitialised ones, say): the planner's sums stay within int32, the
splits within the workspace, and a decode takes such a length as the block table's end without
walking the tiles behind it."""
import math

import pytest
import torch

from mla_paged_kv_03_b200 import binding as B
from mla_paged_kv_03_b200 import workloads as W
from parity_util import assert_lse_close, assert_out_close
from test_gpu_faults import DENSE_SHAPES, dense_gpu, dense_oracle
from test_gpu_shared_prefix import Case

pytestmark = pytest.mark.gpu

MOST = 2 ** 31 - 1


def assert_plan_in_bounds(meta, ns, batch, parts):
    meta, ns = meta.cpu(), ns.cpu()
    steps = ns[1:] - ns[:-1]
    assert ns[0] == 0 and (steps >= 1).all() and ns[-1] <= batch + parts
    live = meta[:, 0] <= meta[:, 2]
    assert live.any()
    assert (meta[live, 0] >= 0).all() and (meta[live, 2] < batch).all()
    assert (meta[live, 1] >= 0).all() and (meta[live, 3] >= 1).all()
    assert (meta[live, 4] >= 0).all() and (meta[live, 4] < steps[meta[live, 0].long()]).all()


@pytest.mark.parametrize("heads", [16, 64, 128])
@pytest.mark.parametrize("lengths", [[MOST] * 40 + [100], [MOST], [100, MOST] * 500,
                                     [5_000_000] * 8192, [MOST - 127] * 33 + [MOST - 128] * 7])
def test_plans_of_far_lengths(heads, lengths):
    B.device_status(reset=True)
    sl = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    meta, ns, parts = B.mla_get_metadata(sl, heads, 1)
    torch.cuda.synchronize()
    assert_plan_in_bounds(meta, ns, len(lengths), parts)
    assert B.device_status() == 0


@pytest.mark.parametrize("heads", [16, 64, 128])
def test_long_lengths_that_fit_are_planned_as_on_the_host(heads):
    # one sequence with more than its share, and a sum below the limit
    lengths = [1 << 28, 70, 0, 1 << 24] + [130] * 300
    meta, ns, parts = B.mla_get_metadata(torch.tensor(lengths, dtype=torch.int32, device="cuda"),
                                         heads, 1)
    hm, hn = B.mla_get_metadata_host(lengths, heads, parts)
    assert torch.equal(meta.cpu(), hm) and torch.equal(ns.cpu(), hn)
    assert B.device_status() == 0


@pytest.mark.parametrize("h_q", [16, 64, 128])
def test_a_sequence_past_its_share_of_the_plan_is_decoded_whole(h_q):
    # 8000 short sequences beside one of 4.6 million tokens, which count for 4.3 million; its pages
    # are few, over and over, so that the softmax is that over one round of them
    B.device_status(reset=True)
    pages, rounds = 16, 4500
    case = W.make_dense([64 * pages, 40], 1, h_q, seed=54, spare_blocks=0)
    bt = torch.zeros((8001, pages * rounds), dtype=torch.int32, device="cuda")
    bt[0] = case.block_table[0].cuda().repeat(rounds)
    bt[1:, 0] = int(case.block_table[1, 0])
    sl = torch.full((8001,), 40, dtype=torch.int32, device="cuda")
    sl[0] = 64 * pages * rounds
    q = case.q[1:].cuda().expand(8001, -1, -1, -1).clone()
    q[0] = case.q[0]
    meta, ns, parts = B.mla_get_metadata(sl, h_q, 1)
    out, lse = B.mla_decode_fwd(q, case.kcache.cuda(), bt, sl, 512, meta, ns, parts,
                                softmax_scale=case.softmax_scale)
    torch.cuda.synchronize()
    assert B.device_status() == 0
    ro, rl = dense_oracle(case)
    rl[0] += math.log(rounds)
    for i in (0, 1, 4000, 8000):
        assert_out_close(out[i:i + 1], ro[min(i, 1):min(i, 1) + 1])
        assert_lse_close(lse[i:i + 1], rl[min(i, 1):min(i, 1) + 1])


@pytest.mark.parametrize("s_q,h_q,d_v", DENSE_SHAPES)
@pytest.mark.parametrize("far", [1 << 20, MOST - 200, MOST])
def test_dense_decode_of_far_lengths(s_q, h_q, d_v, far):
    B.device_status(reset=True)
    case = W.make_dense([700, 130, 64], s_q, h_q, seed=51, d_v=d_v, spare_blocks=1)
    sl = torch.tensor([far, 130, far], dtype=torch.int32)
    bt = case.block_table.clone()
    bt[bt < 0] = 0
    out, lse = dense_gpu(case, bt=bt, sl=sl)
    torch.cuda.synchronize()
    assert B.device_status() >> 16 == B.MLA_DEVERR_BAD_INDEX
    ro, rl = dense_oracle(case, bt=bt, sl=torch.tensor([bt.shape[1] * 64, 130, bt.shape[1] * 64],
                                                       dtype=torch.int32))
    assert_out_close(out, ro)
    assert_lse_close(lse, rl)


@pytest.mark.parametrize("far", [1 << 20, MOST])
@pytest.mark.parametrize("h_q", [16, 128])
def test_shared_prefix_decode_of_far_lengths(h_q, far):
    B.device_status(reset=True)
    c = Case([70, 64, 128], 700, 2, h_q, seed=52)
    t = list(c.dev())
    t[4] = torch.tensor([far, 64, far], dtype=torch.int32, device="cuda")
    c.table[c.table < 0] = 0
    t[3] = c.table.cuda()
    got = c.run(t=t)
    torch.cuda.synchronize()
    assert B.device_status() >> 16 == B.MLA_DEVERR_BAD_INDEX
    c.lengths = [128, 64, 128]
    c.check(got)


@pytest.mark.parametrize("s_q,h_q,d_v", DENSE_SHAPES)
@pytest.mark.parametrize("past", [1, 64, 300, 5000])
def test_a_length_past_the_table_does_not_read_block_0(s_q, h_q, d_v, past):
    # block 0 is nobody's and holds NaN; the splits planned for the tiles past the table are empty
    B.device_status(reset=True)
    case = W.make_dense([640, 130], s_q, h_q, seed=53, d_v=d_v, spare_blocks=2)
    bt = case.block_table
    spare = [i for i in range(case.kcache.shape[0]) if i not in bt.flatten().tolist()]
    if 0 not in spare:
        case.kcache[spare[0]] = case.kcache[0]
        bt[bt == 0] = spare[0]
    case.kcache[0] = float("nan")
    sl = torch.tensor([640 + past, 130], dtype=torch.int32)
    out, lse = dense_gpu(case, bt=bt, sl=sl)
    torch.cuda.synchronize()
    assert B.device_status() >> 16 == B.MLA_DEVERR_BAD_INDEX
    case.kcache[0] = 0
    ro, rl = dense_oracle(case, bt=bt)
    assert_out_close(out, ro)
    assert_lse_close(lse, rl)


@pytest.mark.parametrize("s_q,h_q,d_v", DENSE_SHAPES)
@pytest.mark.parametrize("length", [-1, -64, -1000, -2 ** 31])
def test_a_negative_length_is_an_empty_sequence(s_q, h_q, d_v, length):
    case = W.make_dense([640, 130], s_q, h_q, seed=55, d_v=d_v, spare_blocks=2)
    case.kcache[:] = float("nan")
    sl = torch.tensor([length, length], dtype=torch.int32)
    out, lse = dense_gpu(case, sl=sl)
    torch.cuda.synchronize()
    assert (out == 0).all() and torch.isneginf(lse).all()
    c = Case([0, 0], 0, s_q, h_q, seed=56)
    t = list(c.dev())
    t[1] = torch.full_like(t[1], float("nan"))
    t[4] = sl.cuda()
    c.check(c.run(t=t))

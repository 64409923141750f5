"""Cache rows behind a sequence hold anything: NaN and infinities there change no
bit of any decode over the paged cache."""
import pytest
import torch

from mla_paged_kv_03_b200 import binding as B

pytestmark = pytest.mark.gpu

LENGTHS = [1, 63, 64, 65, 127, 130, 255, 257, 0, 700]


def caches(lengths, extra=(), seed=0, spare=2):
    """(clean cache, the same with NaN and infinities in every row that no sequence has, tables)."""
    g = torch.Generator().manual_seed(seed)
    every = list(lengths) + list(extra)
    pages = [-(-n // 64) for n in every]
    blocks = sum(pages) + spare
    perm = torch.randperm(blocks, generator=g).to(torch.int32)
    cache = torch.randn((blocks, 64, 1, 576), generator=g).to(torch.bfloat16)
    used = torch.zeros((blocks, 64), dtype=torch.bool)
    table = torch.full((len(every), max(1, max(pages))), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(every):
        table[b, :pages[b]] = perm[at:at + pages[b]]
        at += pages[b]
        t = torch.arange(n)
        used[table[b].long()[t // 64], t % 64] = True
    bad = cache.clone()
    junk = torch.tensor([float("nan"), float("inf"), -float("inf")], dtype=torch.bfloat16)
    bad[~used] = junk[torch.randint(0, 3, bad[~used].shape, generator=g)]
    assert not torch.isfinite(bad).all()
    return cache.cuda(), bad.cuda(), table.cuda()


def query(b, s_q, h_q, seed=1):
    g = torch.Generator().manual_seed(seed)
    return torch.randn((b, s_q, h_q, 576), generator=g).to(torch.bfloat16).cuda()


def same(a, b):
    torch.cuda.synchronize()
    assert B.device_status() == 0
    for x, y in zip(a, b):
        assert not torch.isnan(x.float()).any()
        assert torch.equal(x, y)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("s_q,h_q,d_v", [(1, 16, 512), (2, 16, 512), (1, 64, 512), (1, 16, 576),
                                         (1, 128, 512), (2, 100, 512), (3, 128, 576)])
def test_dense(s_q, h_q, d_v, causal):
    clean, bad, table = caches(LENGTHS)
    sl = torch.tensor(LENGTHS, dtype=torch.int32, device="cuda")
    q = query(len(LENGTHS), s_q, h_q)

    def run(cache, parts=None):
        meta, ns, n = B.mla_get_metadata(sl, s_q * h_q, 1, num_sm_parts=parts)
        return B.mla_decode_fwd(q, cache, table, sl, d_v, meta, ns, n, causal=causal)

    same(run(bad), run(clean))
    same(run(bad, 3), run(clean, 3))  # few parts: units of many pages
    empty = run(bad)[0][LENGTHS.index(0)]
    assert (empty == 0).all()


def test_fused():
    clean, bad, table = caches(LENGTHS, seed=2)
    sl = torch.tensor(LENGTHS, dtype=torch.int32, device="cuda")
    q = query(len(LENGTHS), 1, 64)
    gain = torch.ones(576, device="cuda")

    def run(cache):
        meta, ns, n = B.mla_get_metadata(sl, 64, 1)
        return B.mla_fused_norm_rope_attn_rope_cast(q, gain, 1e-6, 1e4, cache, table, sl, meta, ns,
                                                    n)

    same(run(bad), run(clean))


@pytest.mark.parametrize("s_q,h_q", [(1, 16), (2, 16), (1, 128), (3, 100)])
@pytest.mark.parametrize("prefix", [1, 64, 100, 257, 640])
def test_shared_prefix(prefix, s_q, h_q):
    clean, bad, table = caches(LENGTHS, extra=[prefix], seed=3)
    sl = torch.tensor(LENGTHS, dtype=torch.int32, device="cuda")
    q = query(len(LENGTHS), s_q, h_q)

    def run(cache, parts=None):
        meta, ns, n = B.mla_shared_prefix_get_metadata(sl, prefix, s_q * h_q, num_sm_parts=parts)
        return B.mla_shared_prefix_decode_fwd(q, cache, table[-1].contiguous(), prefix,
                                              table[:-1].contiguous(), sl, meta, ns, n)

    same(run(bad), run(clean))
    same(run(bad, 3), run(clean, 3))


@pytest.mark.parametrize("h_q", [16, 64, 128])
def test_page_selected(h_q):
    clean, bad, table = caches(LENGTHS, seed=4)
    sl = torch.tensor(LENGTHS, dtype=torch.int32, device="cuda")
    q = query(len(LENGTHS), 1, h_q)

    def run(cache):
        keys = torch.zeros((cache.shape[0], 576), dtype=torch.int8, device="cuda")
        scales = torch.ones(cache.shape[0], device="cuda")
        B.mla_page_keys_update(cache, table, sl, keys, scales)
        out = B.mla_page_sparse_decode(q, cache, keys, scales, table, sl, 3)
        return out + (keys, scales)

    same(run(bad), run(clean))

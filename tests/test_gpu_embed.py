"""The embedding lookup and its gradient on the GPU (through the C ABI) against their fp64
statements (oracle/layer_oracle.py).

Tolerances.  The lookup multiplies once by the factor (itself rounded to fp32) and rounds once:
half a step of the output's type and two roundings in fp32.  A row of the gradient is a sum in
fp32 of n terms, in any grouping: at most n roundings, and three for the factor, its product
and the addition to what was there, each relative to the sum of the magnitudes.
"""
import math
from concurrent.futures import ThreadPoolExecutor

import pytest
import torch

import linear_attention_sequence_shortconv_b200 as prism
from oracle import layer_oracle as ref

pytestmark = pytest.mark.gpu

HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
U = 2.0 ** -24
DT = {"bf16": torch.bfloat16, "fp32": torch.float32}
ID = {32: torch.int32, 64: torch.int64}


def _gen(seed):
    return torch.Generator().manual_seed(seed)


def _ids(B, T, V, bits, kind, seed=0):
    g = _gen(seed)
    if kind == "one":        # every token names the same row
        ids = torch.full((B, T), V // 2)
    elif kind == "zipf":     # a few rows take most tokens
        ids = (torch.exp(torch.rand((B, T), generator=g, dtype=torch.float64) * math.log(V + 1)) - 1).long().clamp(0, V - 1)
        ids = ids * 7919 % V
    elif kind == "runs":     # runs of 7 .. 9 equal ids: they end around a chunk's border
        n = torch.repeat_interleave(torch.arange(B * T), torch.randint(7, 10, (B * T,), generator=g))[:B * T]
        ids = (n % V).view(B, T)
    else:
        ids = torch.randint(0, V, (B, T), generator=g)
    return ids.to(ID[bits])


CASES = [
    # B, T, V, D, table, dtype, bits, kind, lengths
    (1, 1, 1, 1, "fp32", "fp32", 64, "even", None),
    (1, 1, 5, 8, "bf16", "bf16", 32, "even", None),
    (3, 5, 2, 16, "fp32", "bf16", 64, "even", [5, 0, 2]),
    (2, 300, 1023, 24, "fp32", "bf16", 32, "zipf", [300, 17]),     # ids of ten bits with the sentinel: one pass
    (2, 300, 1024, 768, "fp32", "bf16", 64, "zipf", None),         # eleven bits: two passes
    (4, 1000, 50000, 129, "fp32", "fp32", 64, "zipf", [1000, 999, 1, 0]),
    (1, 4097, 3, 40, "bf16", "bf16", 32, "one", None),
    (2, 4096, 1 << 20, 64, "fp32", "fp32", 32, "even", None),      # 21 bits: three passes
    (5, 1024, 700, 100, "fp32", "bf16", 64, "runs", None),
    (3, 333, 90, 2049, "fp32", "bf16", 32, "zipf", [333, 100, 333]),
    (1, 50, 60, 8192, "bf16", "bf16", 64, "zipf", None),
    (1, 16385, 3000, 16, "fp32", "bf16", 32, "zipf", None),        # more than one pair per thread of the sort
    (8, 16384, 1 << 20, 8, "fp32", "fp32", 64, "zipf", [16384] * 7 + [5]),  # the longest batch sorted in one launch
    (1, 200001, 3000, 16, "fp32", "bf16", 32, "zipf", None),       # longer: sorted by tiles
    (3, 100000, 1 << 20, 8, "fp32", "bf16", 64, "zipf", [100000, 1, 77777]),
    (1, 300000, 1, 8, "bf16", "bf16", 32, "one", None),
    (1, 300001, 2, 16, "fp32", "bf16", 32, "zipf", None),           # thousands of chunks in one run: folded
    (2, 100000, 40, 64, "fp32", "fp32", 64, "zipf", [100000, 99999]),
    (1, 280000, 7, 9, "fp32", "bf16", 32, "zipf", [279999]),
]


@pytest.mark.parametrize("B,T,V,D,table,dtype,bits,kind,lengths", CASES)
def test_lookup_and_gradient_match_fp64(B, T, V, D, table, dtype, bits, kind, lengths):
    ids = _ids(B, T, V, bits, kind)
    w = torch.randn((V, D), generator=_gen(1)).to(DT[table])
    d = torch.randn((B, T, D), generator=_gen(2)).to(DT[dtype])
    lens = None if lengths is None else torch.tensor(lengths, dtype=torch.int32).cuda()
    factor = math.sqrt(D)
    out = prism.embed_fwd(ids.cuda(), w.cuda(), scale=factor, lengths=lens, dtype=DT[dtype])
    want = ref.embed(ids, w.double(), factor, lengths)
    err = (out.double().cpu() - want).abs() - (HALF[DT[dtype]] + 2 * U) * want.abs()
    assert out.dtype == DT[dtype] and err.max() <= 0
    pad = ~ref.valid_rows(lengths, B, T)
    assert not out.cpu()[pad].any()

    keep = ref.valid_rows(lengths, B, T).reshape(-1)
    at, rows = ids.reshape(-1).long()[keep], d.double().view(-1, D)[keep]
    total = factor * torch.zeros(V, D, dtype=torch.float64).index_add_(0, at, rows)
    size = factor * torch.zeros(V, D, dtype=torch.float64).index_add_(0, at, rows.abs())
    n = torch.zeros(V, dtype=torch.float64).index_add_(0, at, torch.ones_like(at, dtype=torch.float64))[:, None]
    got = prism.embed_bwd(ids.cuda(), d.cuda(), V, scale=factor, lengths=lens)
    assert prism.stream_status() == 0
    assert ((got.double().cpu() - total).abs() <= (n + 3) * U * size).all()
    assert not got.cpu()[n[:, 0] == 0].any()

    old = torch.randn((V, D), generator=_gen(3))
    acc = old.cuda()
    assert prism.embed_bwd(ids.cuda(), d.cuda(), V, scale=factor, lengths=lens, d_table=acc, accumulate=True) is acc
    assert ((acc.double().cpu() - total - old.double()).abs() <= (n + 3) * U * (size + old.double().abs())).all()
    assert torch.equal(acc.cpu()[n[:, 0] == 0], old[n[:, 0] == 0])


@pytest.mark.parametrize("kind", ["zipf", "runs", "one"])
@pytest.mark.parametrize("D", [40, 768])
def test_gradient_repeats_bit_for_bit_and_whole_tables_are_written(kind, D):
    ids, V = _ids(4, 777, 500, 64, kind).cuda(), 500
    d = torch.randn((4, 777, D), generator=_gen(5)).bfloat16().cuda()
    first = prism.embed_bwd(ids, d, V)
    dirty = torch.full((V, D), float("nan"), device="cuda")
    ws = torch.full((prism.lib().prism_embed_bwd_workspace_size(4, 777, V, D),), 255, dtype=torch.uint8, device="cuda")
    assert torch.equal(prism.embed_bwd(ids, d, V, d_table=dirty, workspace=ws), first)
    assert torch.equal(prism.embed_bwd(ids, d, V, workspace=ws), first)  # what the first call left there does not matter
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    other = prism.embed_bwd(ids, d, V, stream=s)
    s.synchronize()
    assert torch.equal(other, first)


def test_ids_outside_the_table_and_padding():
    B, T, V, D = 2, 6, 10, 24
    ids = torch.tensor([[0, 10, 9, -1, 3, 3], [1, 2, 1 << 40, 5, 6, 7]])
    w, d = torch.randn((V, D), generator=_gen(1)).cuda(), torch.randn((B, T, D), generator=_gen(2)).cuda()
    bad = (ids < 0) | (ids >= V)
    out = prism.embed_fwd(ids.cuda(), w)
    assert prism.stream_status() == 6  # PRISM_ERR_BOUNDS
    assert not out.cpu()[bad].any()
    clean = torch.where(bad, 0, ids)
    good = prism.embed_fwd(clean.cuda(), w)
    assert torch.equal(out.cpu()[~bad], good.cpu()[~bad])
    got = prism.embed_bwd(ids.cuda(), d, V)
    assert prism.stream_status() == 6
    zeroed = torch.where(bad[..., None], 0.0, d.cpu()).cuda()
    assert torch.equal(got, prism.embed_bwd(clean.cuda(), zeroed, V))
    # behind lengths neither ids nor d_out are looked at
    lens = torch.tensor([1, 2], dtype=torch.int32).cuda()
    d2 = d.clone()
    d2[0, 1:] = d2[1, 2:] = float("nan")
    a = prism.embed_bwd(ids.cuda(), d2, V, lengths=lens)
    prism.embed_fwd(ids.cuda(), w, lengths=lens)
    assert prism.stream_status() == 0 and torch.isfinite(a).all()
    assert a.cpu().any(1).nonzero()[:, 0].tolist() == [0, 1, 2]
    # nothing valid at all
    none = torch.zeros(B, dtype=torch.int32).cuda()
    assert not prism.embed_bwd(ids.cuda(), d, V, lengths=none).any()
    assert not prism.embed_fwd(ids.cuda(), w, lengths=none).any() and prism.stream_status() == 0


def test_a_decoded_token_is_a_row():
    ids = torch.tensor([3, 1, 3], dtype=torch.int32).cuda()
    w, d = torch.randn((5, 768), generator=_gen(1)).cuda(), torch.randn((3, 768), generator=_gen(2)).cuda()
    assert torch.equal(prism.embed_fwd(ids, w, scale=2.0), 2.0 * w[ids.long()])
    g = prism.embed_bwd(ids, d, 5)
    assert torch.equal(g[3], d[0] + d[2]) and torch.equal(g[1], d[1]) and not g[[0, 2, 4]].any()


def test_a_captured_graph_follows_its_inputs():
    V, D = 2000, 96
    ids, d = _ids(4, 500, V, 64, "zipf").cuda(), torch.randn((4, 500, D), generator=_gen(5)).cuda()
    w, lens = torch.randn((V, D), generator=_gen(6)).cuda(), torch.tensor([500, 3, 0, 77], dtype=torch.int32).cuda()
    prism.embed_bwd(ids, d, V, lengths=lens)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, grad = prism.embed_fwd(ids, w, lengths=lens), prism.embed_bwd(ids, d, V, lengths=lens)
    for seed in (7, 8):
        ids.copy_(_ids(4, 500, V, 64, "even", seed))
        lens.copy_(torch.tensor([seed, 500, 499, 0], dtype=torch.int32))
        d.copy_(torch.randn((4, 500, D), generator=_gen(seed)))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, prism.embed_fwd(ids, w, lengths=lens))
        assert torch.equal(grad, prism.embed_bwd(ids, d, V, lengths=lens))


@pytest.mark.parametrize("V,D", [(1, 1), (31, 1), (33, 2), (1000, 3), (4097, 11), (500, 24), (129, 232), (67, 257),
                                 (35, 510), (70, 512), (41, 1025)])
@pytest.mark.parametrize("share", [0.0, 0.02, 0.6, 1.0])
def test_every_row_without_a_token_is_zero_and_no_other(V, D, share):
    rows = torch.randperm(V, generator=_gen(8))[:max(1, int(share * V))]
    ids = rows.repeat(2).view(1, -1)
    dirty = torch.full((V + 1, D), float("nan"), device="cuda")
    d = torch.randint(1, 9, (1, ids.shape[1], D), generator=_gen(9)).float()  # their sums are exact
    got = prism.embed_bwd(ids.cuda(), d.cuda(), V, d_table=dirty[:V])
    want = torch.zeros(V, D).index_add_(0, ids.view(-1), d.view(-1, D))
    assert torch.equal(got.cpu(), want)
    assert dirty[V].isnan().all()


def test_rows_beyond_two_to_the_31_elements():
    # the last rows of a table of 2^31 + 2^24 elements, read and written
    V, D = (1 << 18) + 2048, 8192
    ids = torch.tensor([[V - 1, 0, V - 2, V - 1]]).cuda()
    table = torch.zeros((V, D), dtype=torch.bfloat16, device="cuda")
    table[V - 1], table[V - 2], table[0] = 3.0, 2.0, 1.0
    out = prism.embed_fwd(ids, table)
    assert out[0, :, 0].tolist() == [3.0, 1.0, 2.0, 3.0] and out[0, :, -1].tolist() == [3.0, 1.0, 2.0, 3.0]
    del table
    d = torch.ones((1, 4, D), dtype=torch.bfloat16, device="cuda")
    g = prism.embed_bwd(ids, d, V)
    assert g[V - 1].eq(2).all() and g[V - 2].eq(1).all() and g[0].eq(1).all() and not g[1:V - 2].any()
    assert prism.stream_status() == 0


def test_refusals_name_the_argument():
    ids, w = torch.zeros((2, 3), dtype=torch.int64, device="cuda"), torch.zeros((4, 8), device="cuda")
    with pytest.raises(TypeError, match="ids"):
        prism.embed_fwd(ids.float(), w)
    with pytest.raises(ValueError, match="table"):
        prism.embed_fwd(ids, w[0])
    with pytest.raises(ValueError, match="contiguous"):
        prism.embed_fwd(ids, w.t())
    with pytest.raises(TypeError, match="float16"):
        prism.embed_fwd(ids, w, dtype=torch.float16)
    with pytest.raises(ValueError, match="out"):
        prism.embed_fwd(ids, w, out=torch.zeros((2, 3, 7), device="cuda"))
    with pytest.raises(prism.PrismError, match="UNSUPPORTED"):
        prism.embed_fwd(ids, w.bfloat16(), dtype=torch.float32)
    with pytest.raises(ValueError, match="d_out"):
        prism.embed_bwd(ids, torch.zeros((2, 4, 8), device="cuda"), 4)
    with pytest.raises(ValueError, match="d_table"):
        prism.embed_bwd(ids, torch.zeros((2, 3, 8), device="cuda"), 4, accumulate=True)
    with pytest.raises(prism.PrismError, match="WORKSPACE"):
        prism.embed_bwd(ids, torch.zeros((2, 3, 8), device="cuda"), 4,
                        workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))


def test_sizes_beyond_32_bits_are_refused():
    # a table of 2^32 + 5 rows fits the device, and the C entry points take sizes of 32 bits
    ids, d = torch.zeros((1, 3), dtype=torch.int64, device="cuda"), torch.ones((1, 3, 1), device="cuda")
    with pytest.raises(prism.PrismError, match="UNSUPPORTED"):
        prism.embed_bwd(ids, d, (1 << 32) + 5)
    with pytest.raises(prism.PrismError, match="UNSUPPORTED"):
        prism.embed_fwd(ids[:, :1].expand((1 << 32) + 5, 1), torch.zeros((1, 1), device="cuda"))


@pytest.mark.parametrize("D", [8, 9, 64])
@pytest.mark.parametrize("kind", ["even", "one", "runs"])
def test_subnormal_numbers_are_added_to_and_kept(D, kind):
    # what a named row holds below 2^-126 stays, and so does a sum down there.  All values are
    # multiples of 2^-149 below 2^-126, so that every sum is exact in any order
    V, N = 300, 1500
    ids = _ids(1, N, V, 64, kind)
    tiny = 2.0 ** -149
    old = (torch.randint(-4000, 4000, (V, D), generator=_gen(1)).double() * tiny).float()
    d = (torch.randint(-1000, 1000, (1, N, D), generator=_gen(2)).double() * tiny).float()
    want = old.double().index_add_(0, ids.view(-1), d.double().view(-1, D))
    got = prism.embed_bwd(ids.cuda(), d.cuda(), V, d_table=old.cuda(), accumulate=True)
    assert torch.equal(got.double().cpu(), want)
    dense = prism.embed_bwd(ids.cuda(), d.cuda(), V)
    assert torch.equal(dense.double().cpu(), want - old.double())


@pytest.mark.parametrize("N,V,D,bits", [(8193, 1023, 24, 32), (16384, 1024, 40, 64), (16385, 70000, 8, 32),
                                        (30001, 1 << 20, 16, 64), (32768, 32000, 64, 32)])
def test_without_a_large_cluster_the_gradient_is_the_same(N, V, D, bits):
    # more tokens than eight blocks sort: by tiles where the device has no place for sixteen
    ids, d = _ids(1, N, V, bits, "zipf").cuda(), torch.randn((1, N, D), generator=_gen(2)).cuda()
    lens = torch.tensor([N - 3], dtype=torch.int32).cuda()
    old = torch.randn((V, D), generator=_gen(3))
    runs = []
    try:
        for portable in (False, True):
            prism.set_portable_clusters(portable)
            added = prism.embed_bwd(ids, d, V, lengths=lens, d_table=old.cuda(), accumulate=True)
            runs.append([prism.embed_bwd(ids, d, V), prism.embed_bwd(ids, d, V, lengths=lens), added])
    finally:
        prism.set_portable_clusters(False)
    assert prism.stream_status() == 0
    assert all(torch.equal(a, b) for a, b in zip(*runs))


@pytest.mark.parametrize("N", [16384, 16385, 32768, 32769])
@pytest.mark.parametrize("V,bits", [(900, 32), (30000, 64), (1 << 20, 32)])  # one, two and three passes
def test_gradient_where_the_sort_changes_its_form(N, V, bits):
    # small integers, so that every sum is exact: the last batch with one pair a thread, the last one that
    # a cluster sorts (full), and their successors
    D = 24
    ids = _ids(1, N, V, bits, "zipf").cuda()
    d = torch.randint(-8, 9, (1, N, D), generator=_gen(4)).float().cuda()
    want = torch.zeros((V, D), dtype=torch.float64, device="cuda").index_add_(0, ids.view(-1).long(), d.view(N, D).double())
    assert torch.equal(prism.embed_bwd(ids, d, V).double(), want)
    old = torch.randint(-99, 99, (V, D), generator=_gen(5)).float().cuda()
    got = prism.embed_bwd(ids, d, V, d_table=old.clone(), accumulate=True)
    assert torch.equal(got.double(), want + old) and prism.stream_status() == 0


@pytest.mark.parametrize("V,D,dtype", [(2, 264, "bf16"), (3000, 257, "fp32"), (40, 520, "bf16")])
def test_gradient_of_very_many_tokens_over_several_column_tiles(V, D, dtype):
    # more than 16384 chunks of partial sums, folded and joined for each tile of 256 columns; exact as above
    N = 2_200_003
    gen = torch.Generator(device="cuda").manual_seed(6)
    ids = (torch.rand((1, N), generator=gen, device="cuda") ** 2 * V).int().clamp_(max=V - 1)
    d = torch.randint(0, 4, (1, N, D), generator=gen, device="cuda").to(DT[dtype])
    lens = torch.tensor([N - 7], dtype=torch.int32, device="cuda")
    got = prism.embed_bwd(ids, d, V, lengths=lens)
    want = torch.zeros((V, D), device="cuda")
    for a in range(0, N - 7, 100_000):  # sums below 2^24: exact in any order
        b = min(a + 100_000, N - 7)
        want.index_add_(0, ids[0, a:b], d[0, a:b].float())
    assert want.max() < 2 ** 24 and torch.equal(got, want) and prism.stream_status() == 0
    assert torch.equal(prism.embed_bwd(ids, d, V, lengths=lens), got)


@pytest.mark.parametrize("N,V,D", [(20000, 50000, 40), (70000, 3000, 64), (200000, 1 << 20, 8), (300001, 2, 16),
                                   (300000, 900, 9)])
def test_every_form_of_the_gradient_repeats_bit_for_bit(N, V, D):
    # the cluster, the tiles, the fold and the join of many chunks: twice, from another stream, from a
    # captured graph and from two threads at once
    ids = _ids(1, N, V, 64, "zipf").cuda()
    d = torch.randn((1, N, D), generator=_gen(7)).cuda()
    first = prism.embed_bwd(ids, d, V, scale=1.7)
    again = prism.embed_bwd(ids, d, V, scale=1.7)
    assert torch.equal(first, again)
    torch.cuda.synchronize()

    def other(_):
        s = torch.cuda.Stream()
        out = [prism.embed_bwd(ids, d, V, scale=1.7, stream=s) for _ in range(4)]
        s.synchronize()
        return out

    with ThreadPoolExecutor(2) as pool:
        for outs in pool.map(other, range(2)):
            assert all(torch.equal(t, first) for t in outs)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = prism.embed_bwd(ids, d, V, scale=1.7)
    for _ in range(2):
        out.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, first)
    ids.copy_(_ids(1, N, V, 64, "even", 3))
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, prism.embed_bwd(ids, d, V, scale=1.7)) and prism.stream_status() == 0


@pytest.mark.parametrize("N,V,D", [(3000, 500, 3), (40000, 9000, 8), (300000, 40, 24)])
def test_sums_of_several_calls_add_up(N, V, D):
    # rows that share a sector of the table, call after call; integers, so that every sum is exact
    ids = _ids(1, N, V, 32, "zipf").cuda()
    table, want = torch.zeros((V, D), device="cuda"), torch.zeros((V, D), dtype=torch.float64, device="cuda")
    for k in range(4):
        d = torch.randint(-8, 9, (1, N, D), generator=_gen(k)).float().cuda()
        prism.embed_bwd(ids, d, V, d_table=table, accumulate=True)
        want.index_add_(0, ids.view(-1), d.view(N, D).double())
    assert torch.equal(table.double(), want) and prism.stream_status() == 0

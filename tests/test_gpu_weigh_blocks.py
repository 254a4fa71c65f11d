"""Softmax weights of many query rows on the GPU, in blocks of 128 positions (64 of more than 128 channels), which calls
of many sequences, key heads or positions take, and with more blocks than workgroups.  Against the plain 64-bit
definition, with the tolerances of test_gpu_weigh."""
import numpy as np
import pytest

from tests._util import say
from tests.test_gpu_attention4 import Batch4
from tests.test_gpu_weigh import CACHES, Weights

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def blocks(b, tokens):
    """Blocks of `tokens` positions in as many sequences as the call has, as wide as its table: what the choice goes by."""
    return len(b.seqs) * b.kv * (b.table.shape[1] * b.page / tokens + 1)


def large(b):
    """The batch is one of large blocks (three for every four compute units, at least)."""
    cus = torch.cuda.get_device_properties(0).multi_processor_count
    assert blocks(b, 64 if b.dim > 128 else 128) >= 0.75 * cus
    return b


def widened(b, columns):
    """Its table with room for more pages, which nobody uses."""
    b.table = torch.nn.functional.pad(b.table, (0, columns), value=-1)
    return b


# two of many rows, blocks that begin in the middle of nothing and end after a sequence's end, one kernel's sequences
# between the other's, an idle one
SEQS = [(140, 700), (0, 33), (260, 260), (1, 90), (70, 500), (5, 300)]


@pytest.mark.parametrize("kind,cache", CACHES)
@pytest.mark.parametrize("heads,kv,dim,page", [(16, 8, 64, 16), (16, 8, 80, 32), (8, 8, 96, 16), (16, 8, 128, 64), (16, 8, 112, 16),
                                               (8, 8, 16, 128), (12, 6, 256, 16), (8, 8, 144, 32)])
def test_large_blocks(heads, kv, dim, page, kind, cache):
    say(f"large blocks {heads}/{kv} x {dim}, page {page}, {kind} over {cache}")
    w = Weights(large(Batch4(SEQS, heads, kv, dim, page, kind, cache, seed=dim + heads)))
    w.check(w.run())


@pytest.mark.parametrize("dim,kind,cache", [(128, "bf16", "bf16"), (64, "f16", "e2m1"), (80, "f16", "e4m3"), (256, "bf16", "e2m1")])
@pytest.mark.parametrize("causal,window", [(True, 1), (True, 33), (True, 200), (False, 0), (False, 150)])
def test_masks_in_large_blocks(dim, kind, cache, causal, window):
    """Windows and no causality, more new tokens than positions."""
    say("masks in large blocks", dim, kind, cache, causal, window)
    seqs = [(140, 700), (260, 260), (180, 100), (150, 0), (1, 400)]
    b = large(Batch4(seqs, 8, 8, dim, 16, kind, cache, seed=window + dim))
    w = Weights(b, causal=causal, window=window)
    w.check(w.run())


@pytest.mark.parametrize("cache", ["f16", "e4m3", "e2m1"])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_garbage_beside_large_blocks(dim, cache):
    """Keys that are not finite behind the last position, before the window and in spare pages; rows left out whose
    queries hold anything; weights that are NaN where nobody looks and in new positions."""
    say("garbage beside large blocks", dim, cache)
    seqs, window = [(150, 450), (200, 230), (1, 60)], 90
    b = large(widened(Batch4(seqs, 8, 8, dim, 32, "f16", cache, seed=dim), 40))
    w = Weights(b, window=window)
    out = torch.zeros((b.T, 8), dtype=torch.bool)
    out[3:140:5], out[:, 2] = True, True
    w.lse[out.cuda()] = -float("inf")
    clean = w.run()
    used, new = (torch.zeros((b.pages, 32), dtype=torch.bool) for _ in range(2))
    for i, (n, length) in enumerate(seqs):
        for j in range(length):
            at = (b.table[i, j // 32].long(), j % 32)
            used[at], new[at] = j > length - n - window, j >= length - n
    x = b.tensors[2 if cache == "e2m1" else 0].view(torch.uint8 if cache != "f16" else torch.int16)
    x[~used[:, None].expand(-1, 8, -1).cuda()] = 255 if cache == "e2m1" else 127 if cache == "e4m3" else 0x7E00
    b.q[out.cuda()] = float("nan")
    got = w.run(torch.where((~used | new)[:, None].cuda(), torch.full_like(w.old, float("nan")), w.old))
    seen = used[:, None].expand(-1, 8, -1).cuda()
    assert torch.equal(got[seen], clean[seen]) and torch.isnan(got[~seen]).all()


# (key heads, channels, new tokens, positions, positions of a block)
@pytest.mark.parametrize("kv,dim,n,length,tokens", [(16, 64, 200, 4400, 128), (16, 128, 150, 4370, 128), (8, 256, 140, 4500, 64),
                                                    (8, 64, 200, 2800, 32), (4, 128, 131, 5500, 32)])
@pytest.mark.parametrize("cache", ["f16", "e2m1"])
def test_more_blocks_than_workgroups(kv, dim, n, length, tokens, cache):
    """Workgroups that take several blocks: of one sequence and of two; the same every time."""
    say("several blocks a workgroup", kv, dim, n, length, cache)
    cus = torch.cuda.get_device_properties(0).multi_processor_count
    w = Weights(Batch4([(n, length)], kv, kv, dim, 16, "f16", cache, seed=kv))
    per_head = (length + tokens - 1) // tokens
    assert kv * per_head > 2 * cus and (tokens == 32) == (blocks(w.b, 64 if dim > 128 else 128) < 0.75 * cus)
    got = w.run()
    w.check(got)
    for _ in range(3):
        assert torch.equal(w.run(), got)


def test_a_prompt_among_decoding_sequences():
    """One chunk of a prompt and 63 sequences of one token: blocks by the table's width, most of which nobody has."""
    say("prompt among decoding sequences")
    seqs = [(1, 30 + 11 * i) for i in range(40)] + [(300, 900)] + [(1, 700 - 20 * i) for i in range(23)]
    w = Weights(large(Batch4(seqs, 8, 2, 128, 16, "bf16", "e4m3", seed=1)))
    w.check(w.run())


@pytest.mark.parametrize("columns", [0, 90])
def test_many_rows_past_32_bits(columns):
    """Weights at the end of a pool of more than 2^32 bytes of them, keys past 2^32 bytes, in both sizes of blocks."""
    say("large pool", columns)
    b = widened(Batch4([(150, 200), (30, 90), (260, 300)], 8, 8, 16, 16, "f16", "e2m1", seed=12), columns)
    if columns:
        large(b)
    pages = (2 ** 30 + 2 ** 26) // (8 * 16)
    w = Weights(b)
    small = w.run()
    w.check(small)
    at = pages - b.pages
    big = [torch.empty((pages, *x.shape[1:]), dtype=torch.uint8, device="cuda") for x in b.tensors]
    for x, y in zip(big, b.tensors):
        x[at:] = y
    weight = torch.zeros((pages, 8, 16), device="cuda")
    weight[at:] = w.old
    b.tensors, b.table = big, torch.where(b.table < 0, b.table, b.table + at).to(torch.int32)
    w.run(weight)
    assert torch.equal(weight[at:], small) and not weight[:at].any()


def test_large_blocks_replayed():
    """Captured, then replayed with other lengths, queries and weights, between eager calls of the same batch."""
    say("large blocks replayed")
    import unstructured_sparse_skinny_amd as L
    seqs = [(140, 700), (200, 300), (1, 90), (70, 500)]
    b = large(widened(Batch4(seqs, 8, 8, 128, 16, "bf16", "e2m1", seed=11), 4))
    w = Weights(b)
    weight, cache = w.old.clone(), b.cache()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        L.lscd_cache_weigh(cache, b.q, w.lse, b.start, b.length, b.table, weight)
    for k in range(4):
        b.length.copy_(torch.tensor([n - 37 * k if n > 200 else n for _, n in seqs], dtype=torch.int32))
        b.q.normal_()
        weight.copy_(w.old)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(weight, w.run())

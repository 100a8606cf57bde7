"""Embedding rows of every size class of their stores: kept in the caches,
through the L2, past all caches."""
import pytest

from gpu_helpers import announce
from quantized_decode_gemv_quantize_amd import binding as B

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", [B.F32, B.BF16])
@pytest.mark.parametrize("n", [2001, 20011, 40009])
@pytest.mark.parametrize("ldo", [1003, 1024])
def test_embed_stores(kind, n, ldo):
    """8, 80 and 160 MB, rows of an odd length with a gap that begin inside lines of 128 bytes and at them, read by
    the next launch on the stream; with scales in a replayed graph."""
    import torch
    K, vocab = 1001, 50
    t = torch.float32 if kind == B.F32 else torch.bfloat16
    table = torch.randn(vocab, K, generator=torch.Generator().manual_seed(n)).to(t).to("cuda:0")
    ids = torch.arange(n, device="cuda:0", dtype=torch.int32) * 7 % (vocab + 1) - 1
    out, copy = torch.full((n, ldo), float("nan"), device="cuda:0"), torch.zeros(n, K, device="cuda:0")
    announce(f"embed {n} rows of {K}")
    B.mmvq_embed(table, kind, vocab, K, ids, n, 0.75, out, ldo)
    copy.copy_(out[:, :K])
    want = torch.where((ids >= 0)[:, None], table.float()[ids.clamp(min=0).long()] * 0.75, 0.0)
    assert torch.equal(copy, want) and bool(out[:, K:].isnan().all())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        B.mmvq_embed(table, kind, vocab, K, ids, n, 0.75, out, ldo)
        copy.copy_(out[:, :K])
    for turn in range(3):
        ids.copy_((ids + 5 + turn) % vocab)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(copy, table.float()[ids.long()] * 0.75) and bool(out[:, K:].isnan().all())

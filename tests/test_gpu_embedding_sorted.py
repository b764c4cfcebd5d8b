"""Scaled vocab-parallel embedding and its gradient by sorted tokens (GPU).

Forward: one fp32 product and one rounding, so the bits are known.  Backward: a sum of n fp32 terms is
off by at most n u times the sum of their magnitudes (u = 2^-24), the factor adds one rounding.
"""
import math

import pytest
import torch

import tensor_transformer_layer_way_gb300 as ttl

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
F8 = torch.float64


def _ids(kind, T, V, seed):
    g = torch.Generator().manual_seed(seed)
    if kind == "same":
        return torch.full((T,), V - 1, dtype=torch.int64)
    ids = torch.randint(0, V, (T,), generator=g)
    if kind == "half":
        ids[torch.rand(T, generator=g) < 0.5] = V // 2
    return ids


def _check(ids, dY, scale, dE, V, base=None):
    h = dY.shape[1]
    rows = dY.to(F8)
    ref = torch.zeros(V, h, dtype=F8, device="cuda").index_add_(0, ids, rows) * scale
    mag = torch.zeros(V, h, dtype=F8, device="cuda").index_add_(0, ids, rows.abs()) * abs(scale)
    count = torch.bincount(ids, minlength=V).to(F8)[:, None]
    got = torch.cat(dE).to(F8)
    if base is not None:
        ref, mag = ref + base.to(F8), mag + base.to(F8).abs()
    assert ((got - ref).abs() <= (count + 2) * U * mag).all()
    empty = count[:, 0] == 0
    assert torch.equal(got[empty], ref[empty])


@pytest.mark.parametrize("t,T,h,V", [(1, 1, 8, 1), (2, 37, 64, 96), (8, 257, 256, 8 * 24), (4, 1000, 4096, 4 * 70000)])
@pytest.mark.parametrize("scale", [1.0, 64.0, -0.3])
def test_lookup_bits(t, T, h, V, scale):
    g = torch.Generator().manual_seed(T)
    ids = torch.randint(0, V, (T,), generator=g).cuda()
    E = [torch.randn(V // t, h, device="cuda").to(torch.bfloat16) for _ in range(t)]
    out = ttl.vocab_parallel_embedding_scaled_fwd(ids, E, scale)
    assert ttl.device_status() == 0
    want = (torch.cat(E)[ids].float() * torch.tensor(scale, dtype=torch.float32, device="cuda")).to(torch.bfloat16)
    assert len(out) == t
    for o in out:
        assert torch.equal(o, want)


@pytest.mark.parametrize("kind", ["uniform", "half", "same"])
@pytest.mark.parametrize("t,T,h,V", [(1, 1, 8, 1), (2, 31, 64, 96), (1, 33, 8, 3), (8, 2049, 256, 8 * 24),
                                     (2, 8191, 72, 2 * 30000), (1, 8193, 40, 20), (4, 20000, 16, 4 * 100000),
                                     (1, 70001, 8, 300), (1, 64, 2304, 70), (1, 300, 8, 16777300)])
def test_gradient(t, T, h, V, kind):
    ids = _ids(kind, T, V, T + V).cuda()
    dY = torch.randn(T, h, device="cuda", generator=torch.Generator("cuda").manual_seed(T)).to(torch.bfloat16)
    scale = math.sqrt(h)
    dE = [torch.full((V // t, h), float("nan"), device="cuda") for _ in range(t)]
    ttl.vocab_parallel_embedding_sorted_bwd(ids, dY, scale, dE)
    assert ttl.device_status() == 0
    _check(ids, dY, scale, dE, V)
    base = torch.randn(V, h, device="cuda")
    acc = [b.clone() for b in base.chunk(t)]
    ttl.vocab_parallel_embedding_sorted_bwd(ids, dY, scale, acc, accumulate=True)
    _check(ids, dY, scale, acc, V, base)
    again = [torch.empty_like(e) for e in dE]
    ttl.vocab_parallel_embedding_sorted_bwd(ids, dY, scale, again)
    for a, b in zip(dE, again):
        assert torch.equal(a, b)                                   # the same bits


def test_agrees_with_the_atomic_gradient():
    t, T, h, V = 4, 3000, 128, 4 * 500
    ids = _ids("half", T, V, 1).cuda()
    dY = torch.randn(T, h, device="cuda").to(torch.bfloat16)
    a = [torch.zeros(V // t, h, device="cuda") for _ in range(t)]
    ttl.vocab_parallel_embedding_bwd(ids, dY, a)
    b = [torch.zeros(V // t, h, device="cuda") for _ in range(t)]
    ttl.vocab_parallel_embedding_sorted_bwd(ids, dY, 1.0, b)
    mag = torch.zeros(V, h, device="cuda", dtype=F8).index_add_(0, ids, dY.to(F8).abs())
    assert ((torch.cat(a).to(F8) - torch.cat(b).to(F8)).abs() <= 2 * T * U * mag).all()


def test_ids_out_of_range_are_left_out():
    t, T, h, V = 2, 100, 64, 2 * 20
    ids = _ids("uniform", T, V, 2)
    bad = ids.clone()
    bad[7], bad[50], bad[99] = V, -1, 1 << 40
    keep = torch.ones(T, dtype=torch.bool)
    keep[[7, 50, 99]] = False
    dY = torch.randn(T, h, device="cuda").to(torch.bfloat16)
    dE = [torch.empty(V // t, h, device="cuda") for _ in range(t)]
    ttl.vocab_parallel_embedding_sorted_bwd(bad.cuda(), dY, 2.0, dE)
    assert ttl.device_status() == ttl.TTL_ERR_DEVICE
    _check(ids[keep].cuda(), dY[keep.cuda()], 2.0, dE, V)
    E = [torch.randn(V // t, h, device="cuda").to(torch.bfloat16) for _ in range(t)]
    out = ttl.vocab_parallel_embedding_scaled_fwd(bad.cuda(), E, 2.0)
    assert ttl.device_status() == ttl.TTL_ERR_DEVICE
    assert torch.count_nonzero(out[1][~keep.cuda()]) == 0
    assert torch.equal(out[0][keep.cuda()], (torch.cat(E)[ids[keep].cuda()].float() * 2).to(torch.bfloat16))
    all_bad = torch.full((T,), -5, dtype=torch.int64, device="cuda")
    ttl.vocab_parallel_embedding_sorted_bwd(all_bad, dY, 2.0, dE)
    assert ttl.device_status() == ttl.TTL_ERR_DEVICE
    assert torch.count_nonzero(torch.cat(dE)) == 0


def test_strided_rows_and_no_tokens():
    t, T, h, V = 2, 65, 64, 2 * 20
    ids = _ids("uniform", T, V, 3).cuda()
    wide = torch.randn(T, 3 * h, device="cuda").to(torch.bfloat16)
    dY = wide[:, h:2 * h]
    dE = [torch.empty(V // t, h, device="cuda") for _ in range(t)]
    ttl.vocab_parallel_embedding_sorted_bwd(ids, dY, 1.5, dE)
    _check(ids, dY, 1.5, dE, V)
    ttl.vocab_parallel_embedding_sorted_bwd(ids[:0], dY[:0].contiguous(), 1.5, dE)
    assert torch.count_nonzero(torch.cat(dE)) == 0


def test_gradient_against_differences():
    """The lookup is linear: <dE, W> = sum over tokens of scale dY . W[id], for any W."""
    t, T, h, V = 2, 500, 64, 2 * 37
    ids = _ids("half", T, V, 4).cuda()
    dY = torch.randn(T, h, device="cuda").to(torch.bfloat16)
    dE = [torch.empty(V // t, h, device="cuda") for _ in range(t)]
    ttl.vocab_parallel_embedding_sorted_bwd(ids, dY, 8.0, dE)
    W = torch.randn(V, h, device="cuda", dtype=F8)
    step = 0.5
    E0 = torch.randn(V, h, device="cuda", dtype=F8)
    loss = lambda e: ((E0 + e * W)[ids] * 8.0 * dY.to(F8)).sum()   # noqa: E731
    want = (loss(step) - loss(-step)) / (2 * step)
    size = (W[ids].abs() * dY.to(F8).abs()).sum() * 8.0
    assert ((torch.cat(dE).to(F8) * W).sum() - want).abs() <= (T + 2) * U * size


def test_graph_replay_on_a_side_stream():
    t, T, h, V = 2, 700, 128, 2 * 50
    ids = _ids("half", T, V, 6).cuda()
    dY = torch.randn(T, h, device="cuda").to(torch.bfloat16)
    want = [torch.empty(V // t, h, device="cuda") for _ in range(t)]
    ttl.vocab_parallel_embedding_sorted_bwd(ids, dY, 1.0, want)
    dE = [torch.empty(V // t, h, device="cuda") for _ in range(t)]
    ws = ttl.embedding_sorted_bwd_workspace(t, T, h, V)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=torch.cuda.Stream()):
        ttl.vocab_parallel_embedding_sorted_bwd(ids, dY, 1.0, dE, ws=ws)
    for _ in range(2):
        for e in dE:
            e.fill_(float("nan"))
        graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(want, dE):
        assert torch.equal(a, b)


# Few tokens of few columns: one launch, each CTA a slice of the rows.  The largest of each, one row, one column
# block past a warp's, more tokens of one id than one warp sums alone, slices of one row.
@pytest.mark.parametrize("kind", ["uniform", "half", "same"])
@pytest.mark.parametrize("t,T,h,V", [(1, 1024, 256, 2000), (2, 1000, 72, 2 * 30000), (1, 512, 512, 5), (4, 700, 264, 4 * 1000),
                                     (1, 1024, 8, 65536), (1, 9, 512, 1), (2, 8, 504, 2), (8, 100, 256, 8 * 8192)])
def test_gradient_of_few_tokens(t, T, h, V, kind):
    test_gradient(t, T, h, V, kind)


@pytest.mark.parametrize("T,h", [(700, 64), (2000, 64), (700, 1024)])
def test_strided_rows_and_bad_ids_at_each_size(T, h):
    t, V = 2, 2 * 300
    ids = _ids("half", T, V, T)
    bad = ids.clone()
    keep = torch.rand(T, generator=torch.Generator().manual_seed(1)) < 0.9
    bad[~keep] = V + 5
    dY = torch.randn(T, 3 * h, device="cuda").to(torch.bfloat16)[:, 2 * h:]
    dE = [torch.empty(V // t, h, device="cuda") for _ in range(t)]
    ttl.vocab_parallel_embedding_sorted_bwd(bad.cuda(), dY, 1.5, dE)
    assert ttl.device_status() == ttl.TTL_ERR_DEVICE
    _check(ids[keep].cuda(), dY[keep.cuda()], 1.5, dE, V)
    base = torch.randn(V, h, device="cuda")
    acc = [b.clone() for b in base.chunk(t)]
    ttl.vocab_parallel_embedding_sorted_bwd(bad.cuda(), dY, 1.5, acc, accumulate=True)
    assert ttl.device_status() == ttl.TTL_ERR_DEVICE
    _check(ids[keep].cuda(), dY[keep.cuda()], 1.5, acc, V, base)

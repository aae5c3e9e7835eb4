"""Scratch of the 4-bit attention: a buffer sized for the largest batch serves
the smaller ones."""
import itertools

import pytest
import torch

import compressed_sparse_attention_14_b200 as csa

L = csa._lib
BATCHES = (1, 2, 3, 5, 8, 9, 12, 16, 18, 20, 24, 30, 37, 40, 49, 64, 74, 75, 100, 148, 149, 400)


@pytest.mark.parametrize("H", [1, 16, 17, 32, 33, 64, 65, 128])
@pytest.mark.parametrize("c", [128, 512])
def test_sizes_grow_with_the_call(H, c):
    lens = (1, 64, 100, 200, 256, 257, 512, 1000, 2048)
    for entries, size in ((lens, lambda n, k: L.csa_sparse_mqa_fp4kv_workspace_size(n, H, c, k)),
                          (lens + (8192, 100000), lambda n, k: L.hca_dense_mqa_fp4kv_workspace_size(n, H, c, k)),
                          (lens, lambda n, k: L.csa_decode_fp4kv_workspace_size(n, 4096, H, c, 64, 128, k)),
                          ((64, 3000, 20000), lambda n, N: L.csa_decode_fp4kv_workspace_size(n, N, H, c, 64, 128, 512))):
        sizes = {(n, k): size(n, k) for n, k in itertools.product(BATCHES, entries)}
        for (n, k), b in sizes.items():
            for n2, k2 in ((n, entries[max(entries.index(k) - 1, 0)]), (BATCHES[max(BATCHES.index(n) - 1, 0)], k)):
                assert sizes[n2, k2] <= b, (n2, k2, n, k)


def test_sizes_stay_bounded():
    # at most 148 partial results of 64 heads
    most = 148 * 64 * (512 + 2) * 4 + 512
    assert 0 < L.hca_dense_mqa_fp4kv_workspace_size(65535, 64, 512, 1 << 20) <= most
    assert L.csa_sparse_mqa_fp4kv_workspace_size(1, 64, 512, 512) == 0        # (the splits merge on chip)


@pytest.mark.gpu
@pytest.mark.parametrize("H,c,R", [(64, 512, 64), (40, 256, 32), (128, 128, 0)])
def test_a_buffer_of_the_largest_batch_serves_every_smaller_one(H, c, R):
    """Called without the binding's own scratch: a buffer that is too small is an error."""
    g = torch.Generator().manual_seed(H)
    N, K, top = 3000, 1024, 150
    kv = csa.csa_quantize_kv_fp4(torch.randn(1, N, c, generator=g).to(torch.bfloat16).cuda(), rope_dims=R)
    q = torch.randn(top, H, c, generator=g).to(torch.bfloat16).cuda()
    seq = torch.zeros(top, dtype=torch.int32).cuda()
    sparse = csa.workspace_size("csa_sparse_mqa_fp4kv", top, H, c, K)
    dense = csa.workspace_size("hca_dense_mqa_fp4kv", top, H, c, N)
    ws = torch.empty(max(sparse, dense), dtype=torch.uint8).cuda()
    st = torch.cuda.current_stream().cuda_stream
    for nq in (1, 2, 7, 8, 16, 18, 24, 36, 40, 74, 100, top):
        pos = torch.full((nq,), N, dtype=torch.int32).cuda()
        out, lse = torch.empty_like(q[:nq]), torch.empty(nq, H).cuda()
        for k in (1, 500, 512, K):
            idx = torch.randint(0, N, (nq, k), generator=g, dtype=torch.int32).cuda()
            assert L.csa_sparse_mqa_fp4kv(q.data_ptr(), kv.data_ptr(), idx.data_ptr(), seq.data_ptr(), nq, 1, H, c, R, N, k,
                                          0.0, None, out.data_ptr(), lse.data_ptr(), ws.data_ptr(), sparse, st) == 0
            want = csa.csa_sparse_mqa_fp4kv(q[:nq], kv, idx, seq_of_q=seq[:nq], rope_dims=R)
            assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
        assert L.hca_dense_mqa_fp4kv(q.data_ptr(), kv.data_ptr(), pos.data_ptr(), seq.data_ptr(), nq, 1, H, c, R, N, 1, 0.0,
                                     None, out.data_ptr(), lse.data_ptr(), ws.data_ptr(), dense, st) == 0
        want = csa.hca_dense_mqa_fp4kv(q[:nq], kv, pos, 1, seq_of_q=seq[:nq], rope_dims=R)
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1])

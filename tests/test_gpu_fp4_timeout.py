"""A device wait that runs out in the 4-bit attention or weights (their first
tile withheld by the library's test hook): the call reports CSA_ERR_TIMEOUT, every
role and every CTA of a cluster ends with its copies landed, and the next call
is right."""
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture
def csa():
    import compressed_sparse_attention_14_b200 as m
    yield m
    m.debug_set(0, 0)


def _runs_out(csa, call):
    want = [t.clone() for t in call()]
    csa.poll_status()
    for polls in (1, 40, 600):                              # below and above the polls between looks at the others
        csa.debug_set(polls, csa.CSA_DEBUG_SKIP_FIRST_TILE)
        try:
            call()
            torch.cuda.synchronize()                        # the kernels returned
        finally:
            csa.debug_set(0, 0)
        with pytest.raises(csa.CsaError) as e:
            csa.poll_status()
        assert e.value.code == csa.CSA_ERR_TIMEOUT
        csa.poll_status()                                   # the word was reset
        assert all(torch.equal(a, b) for a, b in zip(call(), want))
        csa.poll_status()


# one CTA walking several queries; two splits that exchange their sums; several in a cluster; many through the workspace;
# rows of whole 32-byte pieces and others, long rotary parts (asynchronous copies)
@pytest.mark.parametrize("nq,H,c,R,k", [(400, 64, 512, 64, 300), (64, 64, 512, 64, 512), (30, 64, 512, 64, 512),
                                        (3, 64, 384, 96, 2048), (36, 64, 256, 32, 1024), (300, 17, 512, 128, 200)])
def test_attention_whose_first_tile_never_comes(csa, nq, H, c, R, k):
    g = torch.Generator().manual_seed(k)
    N = 700
    kv = csa.csa_quantize_kv_fp4(torch.randn(1, N, c, generator=g).to(torch.bfloat16).to(DEV), rope_dims=R)
    q = torch.randn(nq, H, c, generator=g).to(torch.bfloat16).to(DEV)
    idx = torch.randint(0, N, (nq, k), generator=g, dtype=torch.int32).to(DEV)
    seq = torch.zeros(nq, dtype=torch.int32, device=DEV)
    _runs_out(csa, lambda: csa.csa_sparse_mqa_fp4kv(q, kv, idx, seq_of_q=seq, rope_dims=R))


def test_dense_attention_whose_first_tile_never_comes(csa):
    g = torch.Generator().manual_seed(1)
    B, N, H, c = 4, 3000, 64, 512
    kv = csa.csa_quantize_kv_fp4(torch.randn(B, N, c, generator=g).to(torch.bfloat16).to(DEV))
    q = torch.randn(B, H, c, generator=g).to(torch.bfloat16).to(DEV)
    pos = torch.tensor([N, 0, 64, 1700], dtype=torch.int32, device=DEV)         # some splits have nothing
    _runs_out(csa, lambda: csa.hca_decode_fp4kv(q, kv, pos, 1))


# one query block that stays, two head groups, many queries, one tile and several a CTA
@pytest.mark.parametrize("B,T,N,H,c,R", [(16, 1, 3000, 64, 512, 64), (3, 1, 64, 128, 384, 96), (1, 500, 700, 40, 512, 64),
                                         (150, 3, 400, 65, 256, 0)])
def test_weights_whose_first_tile_never_comes(csa, B, T, N, H, c, R):
    g = torch.Generator().manual_seed(T)
    kv = csa.csa_quantize_kv_fp4(torch.randn(B, N, c, generator=g).to(torch.bfloat16).to(DEV), rope_dims=R)
    q = torch.randn(B, T, H, c, generator=g).to(torch.bfloat16).to(DEV)
    lse = torch.full((B, T, H), 6.0, device=DEV)
    pos = torch.randint(0, N + 1, (B, T), generator=g, dtype=torch.int32)
    pos[0, 0] = N
    pos = pos.to(DEV)
    _runs_out(csa, lambda: (csa.hca_entry_weights_fp4kv(q, lse, kv, pos, 1, rope_dims=R),))


def test_weights_of_a_selection_whose_first_tile_never_comes(csa):
    g = torch.Generator().manual_seed(2)
    nq, N, H, c, k = 20, 500, 64, 512, 1000
    kv = csa.csa_quantize_kv_fp4(torch.randn(1, N, c, generator=g).to(torch.bfloat16).to(DEV))
    q = torch.randn(nq, H, c, generator=g).to(torch.bfloat16).to(DEV)
    lse = torch.full((nq, H), 6.0, device=DEV)
    idx = torch.randint(0, N, (nq, k), generator=g, dtype=torch.int32).to(DEV)
    seq = torch.zeros(nq, dtype=torch.int32, device=DEV)
    _runs_out(csa, lambda: (csa.csa_entry_weights_fp4kv(q, lse, kv, idx, seq_of_q=seq),))

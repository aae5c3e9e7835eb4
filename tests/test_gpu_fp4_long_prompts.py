"""The weights of very long prompts: calls whose queries pass a tile of entries
for longer than any one of their waits may take."""
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture
def csa():
    import compressed_sparse_attention_14_b200 as m
    yield m
    m.debug_set(0, 0)


def _case(csa, T, N, H, c, R, B=1):
    """Queries, lse, cache of a call; four different queries in turn, so that a weight is a sum of four terms."""
    g = torch.Generator().manual_seed(T + N)
    kv = csa.csa_quantize_kv_fp4(torch.randn(B, N, c, generator=g).to(torch.bfloat16).to(DEV), rope_dims=R)
    q4 = torch.randn(B, 4, H, c, generator=g).to(torch.bfloat16).to(DEV)
    q = q4.repeat(1, T // 4, 1, 1)
    lse = torch.full((B, T, H), 4.0, device=DEV)
    return q4, q, lse, kv


def _close(w, one, T, H):
    """w: T / 4 times the sums `one` of the four queries. A thread adds the same positive terms, one a query and 64 heads,
    in either call, (T + 4) ceil(H / 64) fp32 additions in all, and the four threads of an entry two more in each."""
    ref = one.double() * (T // 4)
    assert ((w.double() - ref).abs() <= ((T + 4) * -(-H // 64) + 4) * 2.0 ** -24 * ref).all()


def test_queries_that_see_nothing_at_the_end_of_a_prompt(csa):
    """A padded prompt: the last queries see no entry. Finding that once per tile takes some milliseconds here; once per
    query it would hold every wait for a query up that long."""
    T, pad = 1 << 18, (1 << 18) - 256
    q4, q, lse, kv = _case(csa, T, 100, 1, 128, 0)
    pos = torch.full((1, T), 400, dtype=torch.int32, device=DEV)
    pos[:, T - pad:] = 0
    one = csa.hca_entry_weights_fp4kv(q4, lse[:, :4].contiguous(), kv, pos[:, :4].contiguous(), 4, rope_dims=0)
    csa.debug_set(2000)
    w = csa.hca_entry_weights_fp4kv(q, lse, kv, pos, 4, rope_dims=0)
    csa.poll_status()
    _close(w, one, T - pad, 1)


@pytest.mark.parametrize("T,H,c,B", [(16384, 65, 128, 1), (8192, 64, 512, 1), (16384, 16, 384, 2)])
def test_a_tile_may_be_held_longer_than_a_wait(csa, T, H, c, B):
    """Three and more tiles a CTA, each held for all queries: some milliseconds, with waits limited to a fraction of one
    (the built-in limit is 2000 times as long, and a prompt's queries up to 2^18)."""
    N = 148 * 64 * 3 // B
    q4, q, lse, kv = _case(csa, T, N, H, c, 64, B)
    pos = torch.full((B, T), N, dtype=torch.int32, device=DEV)
    one = csa.hca_entry_weights_fp4kv(q4, lse[:, :4].contiguous(), kv, pos[:, :4].contiguous(), 1)
    csa.debug_set(300)
    w = csa.hca_entry_weights_fp4kv(q, lse, kv, pos, 1)
    csa.poll_status()
    _close(w, one, T, H)

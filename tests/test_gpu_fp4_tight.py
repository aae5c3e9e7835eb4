"""The 4-bit attention and weights within the bounds of tests/fp4_bounds.py,
taken per query, head and entry: tight enough to see a single lost, repeated or
wrong entry (tests/test_fp4_bounds.py plants such mistakes)."""
import numpy as np
import pytest
import torch

import oracle
from tests import fp4_bounds as bounds
from tests import test_gpu_fp4 as shared
from tests.parity import host

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module")
def csa():
    import compressed_sparse_attention_14_b200 as m
    return m


@pytest.fixture
def tight(monkeypatch):
    """The shared cases with the bounds of a query, head and entry in the place of one for the whole call."""
    def check(out, lse, q, V, idx, scale, sink, seq):
        bounds.check_attention(host(out), host(lse), host(q), V, idx, scale, sink, seq)
    monkeypatch.setattr(shared, "check_attention", check)


def _params(test, n=-1):
    return test.pytestmark[n].args[1]


@pytest.mark.parametrize("case", _params(shared.test_sparse_attention))
@pytest.mark.parametrize("with_sink", [False, True])
def test_sparse_attention(csa, tight, case, with_sink):
    shared.test_sparse_attention(csa, *case, with_sink)


@pytest.mark.parametrize("case", _params(shared.test_every_split_and_layout) + _params(shared.test_32_heads_a_cta))
def test_every_split_and_layout(csa, tight, case):
    shared.test_every_split_and_layout(csa, *case)


@pytest.mark.parametrize("case", _params(shared.test_dense_attention))
@pytest.mark.parametrize("with_sink", [False, True])
def test_dense_attention(csa, tight, case, with_sink):
    shared.test_dense_attention(csa, *case, with_sink)


@pytest.mark.parametrize("case", _params(shared.test_many_queries_of_any_length))
def test_many_queries_of_any_length(csa, tight, case):
    shared.test_many_queries_of_any_length(csa, *case)


def test_odd_lists(csa, tight):
    shared.test_sparse_attention_odd_lists(csa)


# rotary parts longer than the codes, and nearly all of a row
@pytest.mark.parametrize("nq,H,c,R,k", [(3, 64, 512, 448, 300), (160, 20, 384, 256, 200), (40, 64, 256, 224, 513),
                                        (2, 128, 512, 480, 700)])
def test_long_rotary_parts(csa, tight, nq, H, c, R, k):
    shared.test_every_split_and_layout(csa, max(nq, 3), H, c, R, k, 0)


# one CTA a query, two splits, clusters, the workspace; 16, 32 and 64 heads a CTA
@pytest.mark.parametrize("nq,H,c,R", [(160, 64, 512, 64), (64, 64, 512, 64), (24, 64, 512, 64), (1, 64, 512, 64),
                                      (3, 128, 384, 96), (150, 16, 256, 32), (9, 30, 128, 0)])
@pytest.mark.parametrize("k", [1, 63, 64, 65, 129, 512, 513, 1000, 2048])
def test_equal_logits_count_every_entry(csa, nq, H, c, R, k):
    """Queries of zeros: all weights are equal, lse is the number of entries, the output their mean."""
    N = 2100
    kv, V = shared._rows(csa, N, c, R, 5)
    g = shared._gen(k + nq)
    idx = torch.stack([torch.randperm(N, generator=g)[:k] for _ in range(nq)]).int()
    if nq > 2:
        idx[1, k // 3:] = -1
        idx[2, :k // 2] = -1
    q = torch.zeros(nq, H, c, dtype=torch.bfloat16)
    seq = torch.zeros(nq, dtype=torch.int32, device=DEV)
    out, lse = csa.csa_sparse_mqa_fp4kv(q.to(DEV), kv, idx.to(DEV), seq_of_q=seq, rope_dims=R)
    # (one head's reference serves all: their queries are the same)
    assert torch.equal(out, out[:, :1].expand_as(out)) and torch.equal(lse, lse[:, :1].expand_as(lse))
    bounds.check_attention(host(out[:, :1]), host(lse[:, :1]), host(q[:, :1]), V[None], idx.numpy(), c ** -0.5, None,
                           np.zeros(nq, int))
    w = host(csa.csa_entry_weights_fp4kv(q.to(DEV), lse, kv, idx.to(DEV), seq_of_q=seq, rope_dims=R))
    for t in range(nq):
        live = idx[t].numpy() >= 0
        assert (w[t, ~live] == 0).all()
        if live.any():
            ref, lim = bounds.weights(host(q[t]), host(lse[t]), V[idx[t].numpy()[live]], c ** -0.5)
            assert bounds.outside(w[t, live], ref, lim) <= 1


@pytest.mark.parametrize("lens,N,H,c,R", [([8999, 8192, 8193, 4097, 1, 0, 64, 65], 9000, 64, 512, 64),
                                          ([30000], 30011, 64, 384, 64), ([5000, 4999], 5000, 40, 256, 32),
                                          ([700] * 160, 700, 16, 128, 0)])
def test_equal_logits_of_every_visible_entry(csa, lens, N, H, c, R):
    B = len(lens)
    kv, V = shared._rows(csa, N, c, R, 6)
    kv = kv[None].repeat(B, 1, 1)
    V = np.broadcast_to(V, (B, N, c))
    q = torch.zeros(B, H, c, dtype=torch.bfloat16)
    pos = torch.tensor(lens, dtype=torch.int32)
    out, lse = csa.hca_decode_fp4kv(q.to(DEV), kv, pos.to(DEV), 1, rope_dims=R)
    assert torch.equal(out, out[:, :1].expand_as(out)) and torch.equal(lse, lse[:, :1].expand_as(lse))
    idx = np.where(np.arange(N) < np.array(lens)[:, None], np.arange(N), -1)
    bounds.check_attention(host(out[:, :1]), host(lse[:, :1]), host(q[:, :1]), V, idx, c ** -0.5, None, np.arange(B))
    w = host(csa.hca_entry_weights_fp4kv(q.to(DEV), lse, kv, pos.to(DEV), 1, rope_dims=R))
    for b, n in enumerate(lens):
        assert (w[b, n:] == 0).all()
        if n:
            ref, lim = bounds.weights(host(q[b]), host(lse[b]), V[b, :n], c ** -0.5)
            assert bounds.outside(w[b, :n], ref, lim) <= 1


def _edges(n):
    """The first and last entries of every tile, of the list and around its middle."""
    at = {0, n - 1, n // 2 - 1, n // 2}
    for e in range(0, n, 64):
        at |= {e, min(e + 63, n - 1)}
    return sorted(at)


@pytest.mark.parametrize("N,H,c,R", [(2000, 2, 512, 64), (1029, 64, 128, 32)])
def test_a_query_along_every_entry(csa, N, H, c, R):
    """Each query's weight lies on one entry: its output is that row, whichever the entry is."""
    kv, V = shared._rows(csa, N, c, R, 7)
    q = torch.from_numpy(2 * V).to(torch.bfloat16)[:, None].repeat(1, H, 1)
    seq = torch.zeros(N, dtype=torch.int32, device=DEV)
    pos = torch.full((N,), N, dtype=torch.int32, device=DEV)
    out, lse = csa.hca_dense_mqa_fp4kv(q.to(DEV), kv, pos, 1, seq_of_q=seq, rope_dims=R)
    at = np.arange(N) if H < 8 else np.array(_edges(N))
    for a in range(0, len(at), 64):
        t = at[a:a + 64]
        bounds.check_attention(host(out)[t][:, :1], host(lse)[t][:, :1], host(q)[t][:, :1], V[None],
                               np.tile(np.arange(N), (len(t), 1)), c ** -0.5, None, np.zeros(len(t), int))
    assert torch.equal(out, out[:, :1].expand_as(out))


@pytest.mark.parametrize("per,k", [(64, 512), (18, 1029), (8, 513), (4, 2000), (1, 512), (1, 2048)])
def test_a_query_along_every_edge_of_a_split_list(csa, per, k):
    """The same over lists that are split in two, in clusters and through the workspace: `per` queries a call."""
    H, c, R, N = 64, 512, 64, 2100
    kv, V = shared._rows(csa, N, c, R, 8)
    order = torch.randperm(N, generator=shared._gen(k))[:k]
    at = _edges(k)
    at = (at * per)[:-(-len(at) // per) * per]                                 # whole calls
    seq = torch.zeros(per, dtype=torch.int32, device=DEV)
    for a in range(0, len(at), per):
        rows = order[at[a:a + per]].numpy()
        q = torch.from_numpy(2 * V[rows]).to(torch.bfloat16)[:, None].repeat(1, H, 1)
        idx = order.int()[None].repeat(per, 1)
        out, lse = csa.csa_sparse_mqa_fp4kv(q.to(DEV), kv, idx.to(DEV), seq_of_q=seq)
        bounds.check_attention(host(out)[:, :1], host(lse)[:, :1], host(q)[:, :1], V[None], idx.numpy(), c ** -0.5, None,
                               np.zeros(per, int))
        assert torch.equal(out, out[:, :1].expand_as(out))


# ---------------------------------------------------------------- weights
@pytest.mark.parametrize("nq,B,N,H,c,R,k", _params(shared.test_weights_of_a_selection) + [
    (64, 64, 600, 64, 512, 64, 512), (30, 1, 900, 65, 384, 96, 700)])
def test_weights_of_a_selection(csa, nq, B, N, H, c, R, k):
    kv, V = shared._rows(csa, B * N, c, R, 11)
    kv, V = kv.reshape(B, N, -1), V.reshape(B, N, c)
    g = shared._gen(k)
    q = (2 * torch.randn(nq, H, c, generator=g)).to(torch.bfloat16)
    idx = torch.randint(-N // 4, N, (nq, k), generator=g, dtype=torch.int32)
    seq = (torch.arange(nq) % B).int()
    dev = dict(seq_of_q=seq.to(DEV), rope_dims=R)
    _, lse = csa.csa_sparse_mqa_fp4kv(q.to(DEV), kv, idx.to(DEV), **dev)
    w = host(csa.csa_entry_weights_fp4kv(q.to(DEV), lse, kv, idx.to(DEV), **dev))
    for t in range(nq):
        live = idx[t].numpy() >= 0
        assert (w[t, ~live] == 0).all()
        if not live.any():
            continue
        ref, lim = bounds.weights(host(q[t]), host(lse[t]), V[t % B, idx[t].numpy()[live]], c ** -0.5)
        assert bounds.outside(w[t, live], ref, lim) <= 1


@pytest.mark.parametrize("B,T,N,H,c,R", _params(shared.test_weights_of_every_entry) + [(16, 1, 3000, 64, 512, 64),
                                                                                      (2, 200, 333, 64, 384, 64)])
def test_weights_of_every_entry(csa, B, T, N, H, c, R):
    kv, V = shared._rows(csa, B * N, c, R, 12)
    kv, V = kv.reshape(B, N, -1), V.reshape(B, N, c)
    g = shared._gen(B + T)
    q = (2 * torch.randn(B * T, H, c, generator=g)).to(torch.bfloat16)
    lens = torch.randint(0, N + 1, (B, T), generator=g)
    lens[0, 0] = N
    lens[-1, -1] = 0
    pos = (4 * lens + 3).int().to(DEV)
    seq = torch.arange(B).repeat_interleave(T).int().to(DEV)
    _, lse = csa.hca_dense_mqa_fp4kv(q.to(DEV), kv, pos.flatten(), 4, seq_of_q=seq, rope_dims=R)
    w = host(csa.hca_entry_weights_fp4kv(q.to(DEV).view(B, T, H, c), lse.view(B, T, H), kv, pos, 4, rope_dims=R))
    for b in range(B):
        ref, lim = np.zeros(N), np.zeros(N)
        for t in range(T):
            n = int(lens[b, t])
            r, l = bounds.weights(host(q[b * T + t]), host(lse[b * T + t]), V[b, :n], c ** -0.5)
            ref[:n] += r
            lim[:n] += l
        lim += (T * -(-H // 64) + 4) * 2.0 ** -24 * ref          # the sum over the queries
        assert bounds.outside(w[b], ref, lim + 1e-37) <= 1


def test_every_decode_step_adds_one_per_head(csa):
    """A bounded cache over some steps: what a step adds to the weights is each entry's share, one per head in all for
    a sequence that has entries and nothing for one that has none."""
    B, cap, c, H, m = 3, 20, 512, 64, 2
    g = shared._gen(15)
    kv4 = torch.full((B, cap, 384), 255, dtype=torch.uint8, device=DEV)        # NaN where nothing is stored
    acc = torch.zeros(B, cap, device=DEV)
    n_ent = torch.zeros(B, dtype=torch.int32, device=DEV)
    entry_pos = torch.full((B, cap), -1, dtype=torch.int32, device=DEV)
    for step in range(60):
        pos = torch.tensor([step, step - 30, -1], dtype=torch.int32, device=DEV)   # the last one never has entries
        q = torch.randn(B, H, c, generator=g).to(torch.bfloat16)
        out, lse = csa.hca_decode_fp4kv(q.to(DEV), kv4, n_ent, 1)
        add = host(csa.hca_entry_weights_fp4kv(q.to(DEV), lse, kv4, n_ent, 1))
        before = acc.clone()
        csa.hca_entry_weights_fp4kv(q.to(DEV), lse, kv4, n_ent, 1, acc=acc, out=acc)
        assert torch.equal(acc, before + torch.from_numpy(add).float().to(DEV))
        V = np.nan_to_num(oracle.dequantize_kv_fp4(kv4.cpu().numpy(), c, 64))
        for b, n in enumerate(n_ent.tolist()):
            assert (add[b, n:] == 0).all()
            if n == 0:
                assert lse[b].isneginf().all()
                continue
            ref, lim = bounds.weights(host(q[b]), host(lse[b]), V[b, :n], c ** -0.5)
            assert bounds.outside(add[b, :n], ref, lim) <= 1
            _, true_l, _, lim_l = bounds.attention(host(q[b:b + 1]), V[b:b + 1], np.arange(n)[None], c ** -0.5)
            assert bounds.outside(host(lse[b:b + 1]), true_l, lim_l) <= 1
            assert abs(add[b].sum() - H) <= lim.sum() + 2 * lim_l.sum()
        slot = csa.csa_evict_slot(acc, n_ent, pos, m, cap, entry_pos=entry_pos, recent=3)
        csa.csa_append_kv_fp4(torch.randn(B, c, generator=g).to(torch.bfloat16).to(DEV), slot, kv4)
    assert n_ent.tolist() == [20, 15, 0]

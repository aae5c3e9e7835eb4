"""Eviction by accumulated weight on the GPU. Plans, moves and slots are whole
numbers and copied values: equal to the oracle's."""
import math

import numpy as np
import pytest
import torch

import oracle
from tests.parity import host
from tests.test_gpu_fp4 import check_attention

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module")
def csa():
    import compressed_sparse_attention_14_b200 as m
    return m


def _weights(B, N, seed, kind):
    g = torch.Generator().manual_seed(seed)
    if kind == "ties":
        return torch.randint(0, 4, (B, N), generator=g).float()
    if kind == "equal":
        return torch.zeros(B, N)
    w = torch.exp(3 * torch.randn(B, N, generator=g))
    if kind == "odd":
        w[torch.rand(B, N, generator=g) < 0.1] = math.nan
        w[torch.rand(B, N, generator=g) < 0.1] = math.inf
        w[torch.rand(B, N, generator=g) < 0.1] = -math.inf
        w[torch.rand(B, N, generator=g) < 0.2] = -0.0
        w[torch.rand(B, N, generator=g) < 0.2] = 0.0
        w[torch.rand(B, N, generator=g) < 0.1] *= -1
    return w


def _expected(acc, n_ent, keep, pos, prot):
    B, N = acc.shape
    M = min(keep, N - keep)
    src, dst = np.full((B, M), -1, np.int32), np.full((B, M), -1, np.int32)
    moves, left = np.zeros(B, np.int32), np.zeros(B, np.int32)
    a, p = acc.copy(), None if pos is None else pos.copy()
    for b in range(B):
        mv, left[b] = oracle.evict_plan(acc[b], n_ent[b], keep, None if pos is None else pos[b],
                                        None if prot is None else prot[b])
        moves[b] = len(mv)
        for i, (s, d) in enumerate(mv):
            src[b, i], dst[b, i] = s, d
            a[b, d] = acc[b, s]
            if p is not None:
                p[b, d] = pos[b, s]
        a[b, left[b]:] = 0
        if p is not None:
            p[b, left[b]:] = -1
    return src, dst, moves, left, a, p


@pytest.mark.parametrize("kind", ["plain", "ties", "equal", "odd"])
@pytest.mark.parametrize("N,keep", [(1, 0), (1, 1), (2, 1), (33, 20), (1024, 1000), (3000, 17), (5003, 2501),
                                    (40000, 4001), (70001, 69000)])
def test_plan(csa, kind, N, keep):
    B = 5 if N < 10000 else 2
    acc = _weights(B, N, N + keep, kind)
    n_ent = torch.tensor([N, N + 9, keep, -4, (N + keep) // 2][:B], dtype=torch.int32)
    pos = torch.argsort(torch.rand(B, N, generator=torch.Generator().manual_seed(N)), 1).int()
    for guarded in (False, True):
        prot = torch.tensor([N, N - 5, 0, 0, N // 2][:B], dtype=torch.int32) if guarded else None
        want = _expected(acc.numpy(), n_ent.numpy(), keep, pos.numpy(), None if prot is None else prot.numpy())
        got = csa.csa_evict_plan(acc.to(DEV), n_ent.to(DEV), keep, entry_pos=pos.to(DEV),
                                 protect_from=None if prot is None else prot.to(DEV))
        for name, g, w in zip(("src", "dst", "n_moves", "n_out", "acc", "pos"), got, want):
            np.testing.assert_array_equal(g.cpu().numpy(), w, err_msg=name)
        if not guarded:                                   # without positions the same
            bare = csa.csa_evict_plan(acc.to(DEV), n_ent.to(DEV), keep)
            for g, w in zip(bare[:5], got[:5]):
                np.testing.assert_array_equal(g.cpu().numpy(), w.cpu().numpy())
            assert bare[5] is None


@pytest.mark.parametrize("B,N,keep", [(4, 300, 130), (1, 9000, 40), (70, 64, 63)])
def test_evict_in_place_moves_every_cache(csa, B, N, keep):
    g = torch.Generator().manual_seed(N)
    acc = _weights(B, N, 3, "plain")
    n_ent = torch.randint(0, N + 1, (B,), generator=g, dtype=torch.int32)
    n_ent[0] = N
    pos = torch.arange(N, dtype=torch.int32).repeat(B, 1)
    prot = (n_ent - 8).int()
    kv4 = torch.randint(0, 256, (B, N, 384), generator=g, dtype=torch.uint8)
    keys = torch.randn(B, N, 8, generator=g).to(torch.bfloat16)
    src, dst, moves, left, a, p = _expected(acc.numpy(), n_ent.numpy(), keep, pos.numpy(), prot.numpy())
    w_kv, w_keys = kv4.clone(), keys.clone()
    for b in range(B):
        for i in range(moves[b]):
            w_kv[b, dst[b, i]], w_keys[b, dst[b, i]] = kv4[b, src[b, i]], keys[b, src[b, i]]
    d = [t.to(DEV) for t in (kv4, keys, acc, n_ent, pos)]
    csa.csa_evict(d[:2], d[2], d[3], keep, entry_pos=d[4], protect_from=prot.to(DEV))
    assert torch.equal(d[0].cpu(), w_kv) and torch.equal(d[1].cpu(), w_keys)
    np.testing.assert_array_equal(d[2].cpu().numpy(), a)
    np.testing.assert_array_equal(d[3].cpu().numpy(), left)
    np.testing.assert_array_equal(d[4].cpu().numpy(), p)
    before = [t.clone() for t in d]
    csa.csa_evict(d[:2], d[2], d[3], keep, entry_pos=d[4], protect_from=prot.to(DEV))     # nothing left to cut
    assert all(torch.equal(x, y) for x, y in zip(before, d))


@pytest.mark.parametrize("kind", ["plain", "ties", "odd"])
@pytest.mark.parametrize("B,N,cap,recent,m", [(1, 1, 1, 0, 1), (9, 40, 33, 4, 4), (3, 900, 700, 0, 2), (2, 64, 8, 20, 1)])
def test_slots_step_by_step(csa, kind, B, N, cap, recent, m):
    g = torch.Generator().manual_seed(cap)
    acc = _weights(B, N, 5, kind)
    n_ent = torch.randint(0, cap + 1, (B,), generator=g, dtype=torch.int32)
    n_ent[0] = cap
    pos = torch.randint(0, 30, (B, N), generator=g, dtype=torch.int32)
    ref = [acc.numpy().copy(), n_ent.numpy().copy(), pos.numpy().copy()]
    d = [t.to(DEV) for t in (acc, n_ent, pos)]
    for step in range(3 * m + 2):
        at = torch.tensor([40 * m + step + b for b in range(B)], dtype=torch.int32)
        if B > 2:
            at[2] = -1
        slot = csa.csa_evict_slot(d[0], d[1], at.to(DEV), m, cap, entry_pos=d[2], recent=recent).cpu().numpy()
        for b in range(B):
            t = int(at[b])
            want = -1
            if t >= 0 and (t + 1) % m == 0:
                i, n = (t + 1) // m - 1, ref[1][b]
                want = n
                if n >= cap:
                    want = oracle.evict_order(ref[0][b, :cap], ref[2][b, :cap], i - recent if recent else None)[-1]
                ref[0][b, want], ref[2][b, want] = 0, i
                ref[1][b] = min(n + 1, cap)
            assert slot[b] == want
        for x, y in zip(d, ref):
            np.testing.assert_array_equal(x.cpu().numpy(), y)
        d[0] += torch.rand(B, N, generator=g).to(DEV)
        ref[0] = d[0].cpu().numpy().copy()


def test_a_budgeted_decode_loop(csa):
    """Compression, slot, store, attention and weights together, as a server
    runs them: the cache stays inside its budget, and every step's output is
    the oracle's attention over the entries then in it."""
    B, cap, c, R, H, m, recent = 3, 24, 512, 64, 64, 4, 3
    g = torch.Generator().manual_seed(8)
    bias = torch.randn(2 * m, c, generator=g).to(DEV)
    state = torch.zeros(B, 2 * m, 4 * c, device=DEV)
    staging = torch.zeros(B, 64, c, dtype=torch.bfloat16, device=DEV)          # the step's bf16 entries by index
    kv4 = torch.full((B, cap, 384), 255, dtype=torch.uint8, device=DEV)        # NaN where nothing is stored
    acc = torch.zeros(B, cap, device=DEV)
    n_ent = torch.zeros(B, dtype=torch.int32, device=DEV)
    entry_pos = torch.full((B, cap), -1, dtype=torch.int32, device=DEV)
    one = torch.ones(B, dtype=torch.int32, device=DEV)
    held = [dict() for _ in range(B)]                                          # slot -> entry index
    for step in range(160):
        p = one * step
        q = torch.randn(B, H, c, generator=g).to(torch.bfloat16)
        qd = q.to(DEV)
        out, lse = csa.hca_decode_fp4kv(qd, kv4, n_ent, 1)
        csa.hca_entry_weights_fp4kv(qd, lse, kv4, n_ent, 1, acc=acc, out=acc)
        if step % 40 == 39:
            V = oracle.dequantize_kv_fp4(kv4.cpu().numpy(), c, R)
            idx = np.full((B, cap), -1, np.int32)
            for b in range(B):
                n = len(held[b])
                idx[b, :n] = np.arange(n)
                for s, i in held[b].items():
                    row = oracle.quantize_kv_fp4(staging[b, i].double().cpu().numpy(), R)
                    assert np.array_equal(kv4[b, s].cpu().numpy(), row)
            check_attention(out, lse, q, np.nan_to_num(V), idx, c ** -0.5, None, np.arange(B))
            # every head's weights add up to 1 at every step with entries
            total = host(acc).sum(1)
            assert (total <= H * (step + 1)).all()
        csa.csa_compress_step(torch.randn(B, 4 * c, generator=g).to(DEV), state, bias, p, staging, m)
        before = acc.clone()
        slot = csa.csa_evict_slot(acc, n_ent, p, m, cap, entry_pos=entry_pos, recent=recent)
        entry = (step + 1) // m - 1
        new = staging[:, max(entry, 0)].contiguous()
        csa.csa_append_kv_fp4(new, slot, kv4)
        for b in range(B):
            s = int(slot[b])
            assert (s >= 0) == ((step + 1) % m == 0)
            if s < 0:
                continue
            if len(held[b]) == cap:
                w = {x: float(before[b, x]) for x, i in held[b].items() if i < entry - recent}
                assert float(before[b, s]) == min(w.values()) and s in w
            held[b][s] = entry
        assert int(n_ent.max()) <= cap
    assert n_ent.tolist() == [cap] * B


def test_empty_batches_and_caches(csa):
    i32 = torch.int32
    z = lambda *shape, dt=i32: torch.zeros(shape, dtype=dt, device=DEV)
    assert csa.csa_evict_plan(z(0, 9, dt=torch.float32), z(0), 4)[0].shape == (0, 4)
    out = csa.csa_evict_plan(z(2, 0, dt=torch.float32), z(2) + 5, 0, entry_pos=z(2, 0), protect_from=z(2))
    assert out[0].shape == (2, 0) and (out[2] == 0).all() and (out[3] == 0).all()
    csa.csa_evict_rows(z(2, 0, 32, dt=torch.uint8), z(2, 0), z(2, 0), z(2))
    assert csa.csa_evict_slot(z(0, 9, dt=torch.float32), z(0), z(0), 4, 3).shape == (0,)
    # keep nothing, keep everything: no moves either way
    acc = torch.arange(10, dtype=torch.float32, device=DEV).reshape(2, 5)
    src, dst, moves, n_out, w, _ = csa.csa_evict_plan(acc, z(2) + 5, 0)
    assert src.shape == (2, 0) and (moves == 0).all() and (n_out == 0).all() and (w == 0).all()
    src, dst, moves, n_out, w, _ = csa.csa_evict_plan(acc, z(2) + 5, 5)
    assert src.shape == (2, 0) and (moves == 0).all() and (n_out == 5).all() and torch.equal(w, acc)

"""csa_evict looks at every cache before it writes anything (no GPU: the plan
and the moves are replaced by records of their calls)."""
import numpy as np
import pytest
import torch

import compressed_sparse_attention_14_b200 as csa


class OnGpu:
    """The parts of a CUDA tensor that the checks look at."""
    is_cuda = True

    def __init__(self, *shape, dtype=torch.uint8, device=0, ptr=0x10000, contiguous=True):
        self.shape, self.dtype, self._dev, self._ptr, self._contiguous = torch.Size(shape), dtype, device, ptr, contiguous
        self.device = torch.device("cuda", device)

    def get_device(self):
        return self._dev

    def is_contiguous(self):
        return self._contiguous

    def data_ptr(self):
        return self._ptr

    def element_size(self):
        return torch.empty((), dtype=self.dtype).element_size()


@pytest.fixture
def calls(monkeypatch):
    seen = []
    monkeypatch.setattr(csa, "csa_evict_plan", lambda *a, **k: seen.append("plan") or (None,) * 6)
    monkeypatch.setattr(csa, "csa_evict_rows", lambda cache, *a: seen.append(tuple(cache.shape)))
    return seen


GOOD = OnGpu(2, 64, 384)


@pytest.mark.parametrize("bad", [
    OnGpu(2, 64, dtype=torch.float32),                     # a scale an entry: rows of 4 bytes
    OnGpu(2, 64, 3, dtype=torch.float32),                  # rows of 12
    OnGpu(2, 64, 0),
    OnGpu(2, 63, 384), OnGpu(2, 128, 384), OnGpu(3, 64, 384),   # not the weights' sequences and entries
    OnGpu(128, 384), OnGpu(64),
    OnGpu(2, 64, 384, contiguous=False), OnGpu(2, 64, 384, device=1), OnGpu(2, 64, 384, ptr=0x10008),
    torch.zeros(2, 64, 384, dtype=torch.uint8)])
def test_a_bad_cache_is_refused_before_the_plan(calls, bad):
    acc = OnGpu(2, 64, dtype=torch.float32)
    for caches in ([bad], [GOOD, bad], [bad, GOOD], (x for x in (GOOD, GOOD, bad))):
        with pytest.raises(ValueError, match="caches"):
            csa.csa_evict(caches, acc, None, 8)
        assert calls == []


def test_good_caches_move_after_the_plan(calls):
    keys = OnGpu(2, 64, 8, dtype=torch.bfloat16)
    csa.csa_evict((x for x in (GOOD, keys)), OnGpu(2, 64, dtype=torch.float32), None, 8)
    assert calls == ["plan", (2, 64, 384), (2, 64, 8)]
    csa.csa_evict([], OnGpu(2, 64, dtype=torch.float32), None, 8)
    assert calls[3:] == ["plan"]


@pytest.mark.gpu
def test_a_refused_eviction_changes_nothing():
    g = torch.Generator().manual_seed(4)
    B, N, keep = 3, 80, 30
    acc = torch.rand(B, N, generator=g).cuda()
    n_ent = torch.tensor([N, 40, 7], dtype=torch.int32).cuda()
    pos = torch.arange(N, dtype=torch.int32).repeat(B, 1).cuda()
    kv4 = torch.randint(0, 256, (B, N, 384), generator=g, dtype=torch.uint8).cuda()
    state = [acc, n_ent, pos, kv4]
    before = [t.clone() for t in state]
    for bad in (torch.ones(B, N, device="cuda"), kv4[:, :N - 1].contiguous(), torch.zeros(B, 2 * N, 384, device="cuda"),
                torch.zeros(B, N, 768, dtype=torch.uint8, device="cuda")[..., ::2], kv4.cpu()):
        with pytest.raises(ValueError, match="caches"):
            csa.csa_evict([kv4, bad], acc, n_ent, keep, entry_pos=pos)
        assert all(torch.equal(a, b) for a, b in zip(state, before))
    csa.csa_evict([kv4], acc, n_ent, keep, entry_pos=pos)
    assert n_ent.tolist() == [30, 30, 7] and not torch.equal(kv4, before[3])
    for b, n in enumerate((30, 30, 7)):                    # a row is where its position says
        assert torch.equal(kv4[b, :n], before[3][b, pos[b, :n].long()])


@pytest.mark.gpu
def test_the_newest_entries_by_position_stay_after_slots_were_reused():
    """A cache whose slots have been reused holds positions far above its slots' numbers: the newest are protected by
    position, as the readme has it, and the others go by weight."""
    g = torch.Generator().manual_seed(6)
    B, N, cap, newest, keep = 2, 64, 50, 12, 30
    acc = torch.rand(B, N, generator=g).cuda()
    n_ent = torch.zeros(B, dtype=torch.int32).cuda()
    pos = torch.full((B, N), -1, dtype=torch.int32).cuda()
    for step in range(400):
        csa.csa_evict_slot(acc, n_ent, torch.full((B,), step, dtype=torch.int32).cuda(), 1, cap, entry_pos=pos, recent=20)
        acc += torch.rand(B, N, generator=g).cuda()
    weight = {(b, int(pos[b, i])): float(acc[b, i]) for b in range(B) for i in range(cap)}
    csa.csa_evict([], acc, n_ent, keep, entry_pos=pos, protect_from=pos.amax(1) - (newest - 1))
    for b in range(B):
        left = set(pos[b, :keep].tolist())
        new = set(range(400 - newest, 400))
        held = {p: w for (x, p), w in weight.items() if x == b and p not in new}
        assert new <= left and left - new == set(sorted(held, key=held.get)[-(keep - newest):])
        assert (pos[b, keep:] == -1).all()


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["plain", "ties", "odd"])
@pytest.mark.parametrize("N,keep", [(393_217, 100_000), (500_003, 499_000), (800_000, 17)])
def test_plans_of_caches_whose_keys_do_not_fit_on_chip(kind, N, keep):
    from tests.test_gpu_evict import _expected, _weights
    acc = _weights(2, N, keep, kind)
    n_ent = torch.tensor([N, N - 12_345], dtype=torch.int32)
    pos = torch.argsort(torch.rand(2, N, generator=torch.Generator().manual_seed(N)), 1).int()
    prot = torch.tensor([N - 9, N // 2], dtype=torch.int32)
    want = _expected(acc.numpy(), n_ent.numpy(), keep, pos.numpy(), prot.numpy())
    got = csa.csa_evict_plan(acc.cuda(), n_ent.cuda(), keep, entry_pos=pos.cuda(), protect_from=prot.cuda())
    for g, w in zip(got, want):
        np.testing.assert_array_equal(g.cpu().numpy(), w)


@pytest.mark.gpu
def test_a_captured_step_of_a_bounded_cache_replays():
    """Weights, slot, store and an eviction in one graph, replayed step by step against the eager calls."""
    B, cap, c, H = 3, 40, 512, 64
    def start():
        return [torch.zeros(B, cap).cuda(), torch.zeros(B, dtype=torch.int32).cuda(),
                torch.full((B, cap), -1, dtype=torch.int32).cuda(), torch.full((B, cap, 384), 255, dtype=torch.uint8).cuda()]
    q = torch.empty(B, H, c, dtype=torch.bfloat16).cuda()
    new = torch.empty(B, c, dtype=torch.bfloat16).cuda()
    pos = torch.zeros(B, dtype=torch.int32).cuda()
    prot = torch.zeros(B, dtype=torch.int32).cuda()

    def step(acc, n_ent, at, kv):
        out, lse = csa.hca_decode_fp4kv(q, kv, n_ent, 1)
        csa.hca_entry_weights_fp4kv(q, lse, kv, n_ent, 1, acc=acc, out=acc)
        csa.csa_evict([kv], acc, n_ent, cap - 8, entry_pos=at, protect_from=prot)
        slot = csa.csa_evict_slot(acc, n_ent, pos, 1, cap - 4, entry_pos=at, recent=2)
        csa.csa_append_kv_fp4(new, slot, kv)
        return out, lse, slot

    eager, held = start(), start()
    q.zero_(), new.zero_()
    step(*start())                                          # (the kernels are loaded)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step(*held)
    g = torch.Generator().manual_seed(9)
    for t in range(120):
        q.copy_(torch.randn(B, H, c, generator=g))
        new.copy_(torch.randn(B, c, generator=g))
        pos.fill_(t)
        prot.fill_(t - 5)
        want = step(*eager)
        graph.replay()
        for a, b in zip((*want, *eager), (*outs, *held)):
            assert torch.equal(a, b)
    assert eager[1].tolist() == [cap - 7] * B

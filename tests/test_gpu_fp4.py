"""The 4-bit KV cache on the GPU against the 64-bit oracle.

* Stored rows are integer decisions: equal to the oracle's, byte for byte, and
  the values read back are equal.
* Attention: the products of stored values and queries are exact in the
  tensor cores, so a logit is off by the rounding of a sum of c terms, at most
  dz = c * 2^-24 * scale * sum_d |q_d v_d|. The softmax weight e^z then carries
  dz, the exponential and the sums 2^-19, and its rounding to bf16 half a step
  (2^-8); the output half a step of its own:
      |out - ref| <= (2^-8 + 2 dz + 2^-19) * sum_s p_s |v_s| + 2^-8 |ref|
      |lse - ref| <= dz + 2^-19 (1 + |ref|)
* Weights: sum_h e^(z - lse), each term off by dz and the exponential:
      |w - ref| <= (e^dz - 1 + 2^-18) * ref
"""
import math

import numpy as np
import pytest
import torch

import oracle
from tests.parity import host

pytestmark = pytest.mark.gpu
DEV = "cuda"
H_, S_ = 2.0 ** -8, 2.0 ** -19


@pytest.fixture(scope="module")
def csa():
    import compressed_sparse_attention_14_b200 as m
    return m


def _gen(seed):
    return torch.Generator().manual_seed(seed)


def _rows(csa, n, c, R, seed, scale=1.0):
    """n packed rows on the GPU and their values in 64 bits."""
    x = (torch.randn(n, c, generator=_gen(seed)) * scale).to(torch.bfloat16)
    packed = csa.csa_quantize_kv_fp4(x.to(DEV), rope_dims=R)
    return packed, oracle.dequantize_kv_fp4(packed.cpu().numpy(), c, R)


def _logit_slack(q, V, scale):
    return q.shape[-1] * 2.0 ** -24 * scale * float((np.abs(q).max((0, 1)) * np.abs(V[np.isfinite(V).all(-1)]).max(
        tuple(range(V.ndim - 2)) if V.ndim > 2 else 0).max(0)).sum()) if V.size else 0.0


def check_attention(out, lse, q, V, idx, scale, sink, seq):
    """out, lse against the oracle over idx [nq, k] (-1: empty), V [B, N, c] float64."""
    q = host(q)
    ref, ref_l = oracle.sparse_mqa(q, V, idx, scale, sink=sink, seq=seq)
    absref, _ = oracle.sparse_mqa(q, V, idx, scale, sink=sink, seq=seq)
    # sum_s p_s |v_s|, from the oracle's own weights
    for t in range(q.shape[0]):
        s = idx[t][idx[t] >= 0]
        if len(s) == 0 or seq[t] < 0:
            absref[t] = 0
            continue
        p = np.exp(scale * (q[t] @ V[seq[t], s].T) - ref_l[t][:, None])
        absref[t] = p @ np.abs(V[seq[t], s])
    dz = _logit_slack(q, V, scale)
    got, gl = host(out), host(lse)
    lim = (H_ + 2 * dz + S_) * absref + H_ * np.abs(ref) + 1e-37
    worst = (np.abs(got - ref) / lim).max()
    assert worst <= 1, f"out {worst:.2f} of the bound"
    fin = np.isfinite(ref_l)
    assert np.array_equal(gl[~fin], ref_l[~fin])
    if fin.any():
        lw = (np.abs(gl[fin] - ref_l[fin]) / (dz + S_ * (1 + np.abs(ref_l[fin])))).max()
        assert lw <= 1, f"lse {lw:.2f} of the bound"


def check_weights(w, ref, dz):
    w = host(w)
    lim = (math.expm1(dz) + 2.0 ** -18) * ref + 1e-37
    assert (np.abs(w - ref) <= lim).all(), f"{(np.abs(w - ref) / lim).max():.2f} of the bound"


# ---------------------------------------------------------------- storage
@pytest.mark.parametrize("c,R", [(512, 64), (512, 0), (384, 96), (256, 32), (128, 96), (128, 0)])
@pytest.mark.parametrize("n", [1, 7, 130])
def test_rows_equal_the_oracles(csa, c, R, n):
    g = _gen(n + c + R)
    x = torch.randn(n, c, generator=g) * torch.exp(15 * torch.randn(n, 1, generator=g))
    if n > 7:
        x[0] = 0
        x[1] = torch.randint(-24, 25, (c,), generator=g) * 0.25       # ties of every kind
        x[1, :16] = 0
        x[1, 0] = 6
        x[2] *= torch.exp(8 * torch.randn(c, generator=g))             # blocks binades apart
        x[3] = 3.3895e38
        x[4] = 1e-39                                                   # bf16 subnormals
        x[5] = -0.0
        x[6, 3] = math.inf
        x[7, c - R - 1] = math.nan
        x[8, 16:] = 0
        for i in range(9, 40):                                         # every step of the scale's mantissa and its ties
            x[i, ::16] = 6 * (1 + (i - 9) / 32)
    x = x.to(torch.bfloat16)
    packed = csa.csa_quantize_kv_fp4(x.to(DEV), rope_dims=R)
    ref = oracle.quantize_kv_fp4(x.double().numpy(), R)
    assert np.array_equal(packed.cpu().numpy(), ref)
    val = csa.csa_dequantize_kv_fp4(packed, c, rope_dims=R)
    np.testing.assert_array_equal(val.double().cpu().numpy(), oracle.dequantize_kv_fp4(ref, c, R))


def test_any_bytes_read_back(csa):
    # every code under every scale byte
    c, R = 256, 0
    rows = np.zeros((256, oracle.fp4_row_bytes(c, R)), np.uint8)
    rows[:, :128] = np.arange(128, dtype=np.uint8) * 2 + np.arange(256)[:, None] % 2
    rows[:, 128:144] = (np.arange(16)[None] * 16 + np.arange(256)[:, None]) % 256
    rows[:, 144] = 33 + np.arange(256) % 190
    val = csa.csa_dequantize_kv_fp4(torch.from_numpy(rows).to(DEV), c, rope_dims=R)
    np.testing.assert_array_equal(val.double().cpu().numpy(), oracle.dequantize_kv_fp4(rows, c, R))


@pytest.mark.parametrize("c,R,n", [(512, 64, 1), (512, 64, 35), (384, 32, 18), (128, 64, 67)])
@pytest.mark.parametrize("shift", [0, 8, 16])
def test_rows_at_any_16_byte_address(csa, c, R, n, shift):
    x = torch.randn(n * c + 32, generator=_gen(n)).to(torch.bfloat16).to(DEV)
    rows = x[shift:shift + n * c].view(n, c)
    rb = csa.csa_fp4_row_bytes(c, R)
    room = torch.full((n * rb + 64,), 9, dtype=torch.uint8, device=DEV)
    packed = csa.csa_quantize_kv_fp4(rows, rope_dims=R, out=room[2 * shift:2 * shift + n * rb].view(n, rb))
    ref = oracle.quantize_kv_fp4(rows.double().cpu().numpy(), R)
    assert np.array_equal(packed.cpu().numpy(), ref)
    assert (room[:2 * shift] == 9).all() and (room[2 * shift + n * rb:] == 9).all()
    back = torch.full((n * c + 32,), -3.0, dtype=torch.bfloat16, device=DEV)
    csa.csa_dequantize_kv_fp4(packed, c, rope_dims=R, out=back[shift:shift + n * c].view(n, c))
    assert np.array_equal(host(back[shift:shift + n * c].view(n, c)), oracle.dequantize_kv_fp4(ref, c, R))
    assert (back[:shift] == -3).all() and (back[shift + n * c:] == -3).all()


@pytest.mark.parametrize("B,c,R", [(1, 512, 64), (65, 256, 32), (40, 128, 0)])
def test_append_writes_its_slot_only(csa, B, c, R):
    N = 5
    rb = csa.csa_fp4_row_bytes(c, R)
    cache = torch.full((B, N, rb), 7, dtype=torch.uint8, device=DEV)
    x = torch.randn(B, c, generator=_gen(B)).to(torch.bfloat16)
    slot = torch.arange(B, dtype=torch.int32) % (N + 2) - 1            # -1 .. N
    csa.csa_append_kv_fp4(x.to(DEV), slot.to(DEV), cache, rope_dims=R)
    ref = np.full((B, N, rb), 7, np.uint8)
    for b in range(B):
        if 0 <= slot[b] < N:
            ref[b, slot[b]] = oracle.quantize_kv_fp4(x[b].double().numpy(), R)
    assert np.array_equal(cache.cpu().numpy(), ref)


# ---------------------------------------------------------------- attention over a selection
@pytest.mark.parametrize("nq,B,N,H,c,R,k", [
    (1, 1, 1, 1, 128, 0, 1), (3, 3, 300, 64, 512, 64, 512), (2, 2, 200, 128, 512, 64, 129), (5, 2, 90, 24, 256, 32, 37),
    (4, 4, 140, 65, 384, 96, 128), (3, 3, 260, 64, 512, 0, 1000), (2, 1, 2500, 100, 128, 96, 2048),
    (9, 9, 64, 8, 512, 64, 256), (160, 1, 200, 64, 512, 64, 384)])
@pytest.mark.parametrize("with_sink", [False, True])
def test_sparse_attention(csa, nq, B, N, H, c, R, k, with_sink):
    kv, V = _rows(csa, B * N, c, R, 3)
    kv, V = kv.reshape(B, N, -1), V.reshape(B, N, c)
    g = _gen(k)
    q = (2 * torch.randn(nq, H, c, generator=g)).to(torch.bfloat16)
    idx = torch.randint(0, N, (nq, k), generator=g, dtype=torch.int32)          # repeats too
    idx[torch.rand(nq, k, generator=g) < 0.3] = -1
    if nq > 1:
        idx[1] = -1                                                              # nothing selected
    if k > 200:
        idx[0, :130] = -1                                                        # an empty first tile
    seq = None if B == nq else torch.arange(nq, dtype=torch.int32) % B
    sink = torch.randn(H, generator=g) if with_sink else None
    # unread rows hold NaN: an empty slot must not touch the row it might default to
    used = torch.zeros(B, N, dtype=torch.bool)
    for t in range(nq):
        used[t % B, idx[t][idx[t] >= 0].long()] = True
    kv[~used.to(DEV)] = 255
    out, lse = csa.csa_sparse_mqa_fp4kv(q.to(DEV), kv, idx.to(DEV), rope_dims=R,
                                        sink=None if sink is None else sink.to(DEV),
                                        seq_of_q=None if seq is None else seq.to(DEV))
    ids = idx.numpy().copy()
    V = np.where(used.numpy()[..., None], V, 0)
    check_attention(out, lse, q, V, ids, 1 / math.sqrt(c), None if sink is None else sink.double().numpy(),
                    np.arange(nq) % B)
    again, lse2 = csa.csa_sparse_mqa_fp4kv(q.to(DEV), kv, idx.to(DEV), rope_dims=R,
                                           sink=None if sink is None else sink.to(DEV),
                                           seq_of_q=None if seq is None else seq.to(DEV))
    assert torch.equal(out, again) and torch.equal(lse, lse2)


# heads per CTA 16 and 64; one, two, several and many splits of a query; rows of whole 32-byte pieces and others, at
# any 16-byte address
@pytest.mark.parametrize("nq,H,c,R,k,shift", [
    (64, 64, 512, 64, 512, 0), (64, 64, 512, 64, 512, 16), (64, 40, 384, 64, 500, 0), (30, 64, 512, 64, 512, 0),
    (20, 65, 256, 64, 600, 0), (20, 33, 384, 96, 640, 16), (36, 64, 512, 64, 1024, 0), (36, 64, 384, 96, 1024, 0),
    (160, 17, 384, 64, 300, 0), (8, 64, 384, 64, 512, 32), (3, 128, 512, 0, 1024, 0), (150, 16, 512, 64, 700, 16)])
def test_every_split_and_layout(csa, nq, H, c, R, k, shift):
    N, rb = 400, csa.csa_fp4_row_bytes(c, R)
    rows, V = _rows(csa, 3 * N, c, R, 60)
    flat = torch.zeros(3 * N * rb + 64, dtype=torch.uint8, device=DEV)
    kv = flat[shift:shift + 3 * N * rb].view(3, N, rb)
    kv.copy_(rows.view(3, N, rb))
    g = _gen(nq + k)
    q = (2 * torch.randn(nq, H, c, generator=g)).to(torch.bfloat16)
    idx = torch.randint(-N // 8, N, (nq, k), generator=g, dtype=torch.int32)
    idx[0, 64:] = -1                                                             # later splits see nothing
    idx[1, :-70] = -1                                                            # and earlier ones
    idx[2] = -1
    seq = torch.arange(nq, dtype=torch.int32) % 3
    sink = torch.randn(H, generator=g)
    out, lse = csa.csa_sparse_mqa_fp4kv(q.to(DEV), kv, idx.to(DEV), rope_dims=R, sink=sink.to(DEV),
                                        seq_of_q=seq.to(DEV))
    ids = idx.numpy().copy()
    ids[ids < 0] = -1
    check_attention(out, lse, q, V.reshape(3, N, c), ids, c ** -0.5, sink.double().numpy(), seq.numpy())
    w = csa.csa_entry_weights_fp4kv(q.to(DEV), lse, kv, idx.to(DEV), rope_dims=R, seq_of_q=seq.to(DEV))
    ref = oracle.entry_weights(host(q), host(lse), V.reshape(3, N, c), ids, c ** -0.5, seq.numpy())
    check_weights(w, ref, _logit_slack(host(q), V.reshape(3, N, c), c ** -0.5))


# 32 heads per CTA: unsplit, in two, several and many splits, more queries than SMs
@pytest.mark.parametrize("nq,H,c,R,k,shift", [
    (60, 64, 512, 64, 200, 0), (30, 64, 512, 64, 256, 16), (20, 100, 256, 32, 256, 0), (21, 128, 384, 64, 130, 0),
    (5, 24, 512, 64, 1500, 0), (3, 32, 128, 96, 2048, 0), (12, 17, 384, 96, 700, 16), (400, 30, 512, 64, 300, 0),
    (200, 32, 256, 0, 100, 0)])
def test_32_heads_a_cta(csa, nq, H, c, R, k, shift):
    test_every_split_and_layout(csa, nq, H, c, R, k, shift)


def test_dense_attention_of_32_heads(csa):
    test_dense_attention(csa, 9000, 32, 512, 64, [9000, 130], True)
    test_dense_attention(csa, 500, 20, 384, 96, [500, 0, 64, 65], False)


# more queries than SMs: a CTA goes from one query to the next, of any number of tiles
@pytest.mark.parametrize("nq,B,N,H,c,R", [(700, 3, 150, 72, 256, 64), (500, 2, 330, 20, 512, 64), (401, 4, 70, 64, 384, 64),
                                          (450, 1, 129, 16, 384, 96)])
def test_many_queries_of_any_length(csa, nq, B, N, H, c, R):
    kv, V = _rows(csa, B * N, c, R, 50)
    kv, V = kv.reshape(B, N, -1), V.reshape(B, N, c)
    g = _gen(nq)
    q = (3 * torch.randn(nq, H, c, generator=g)).to(torch.bfloat16)
    pos = torch.randint(0, 4 * N + 40, (nq,), generator=g, dtype=torch.int32)
    pos[torch.rand(nq, generator=g) < 0.2] = 3                                   # nothing visible
    pos[:149] = 0                                                                # a first round of nothing
    pos[300:] = 4 * N
    seq = torch.randint(0, B, (nq,), generator=g, dtype=torch.int32)
    seq[-1] = B                                                                  # no such sequence
    sink = torch.randn(H, generator=g)
    out, lse = csa.hca_dense_mqa_fp4kv(q.to(DEV), kv, pos.to(DEV), 4, seq_of_q=seq.to(DEV), sink=sink.to(DEV),
                                       rope_dims=R)
    idx = np.full((nq, N), -1, np.int32)
    for t in range(nq - 1):
        n = min(N, max(0, int(pos[t])) // 4)
        idx[t, :n] = np.arange(n)
    check_attention(out, lse, q, V, idx, c ** -0.5, sink.double().numpy(), np.minimum(seq.numpy(), B - 1))
    again, lse2 = csa.hca_dense_mqa_fp4kv(q.to(DEV), kv, pos.to(DEV), 4, seq_of_q=seq.to(DEV), sink=sink.to(DEV),
                                          rope_dims=R)
    assert torch.equal(out, again) and torch.equal(lse, lse2)
    # and as a selection
    lists = torch.from_numpy(idx).to(DEV)
    sel, lse3 = csa.csa_sparse_mqa_fp4kv(q.to(DEV), kv, lists, seq_of_q=seq.to(DEV), sink=sink.to(DEV), rope_dims=R)
    check_attention(sel, lse3, q, V, idx, c ** -0.5, sink.double().numpy(), np.minimum(seq.numpy(), B - 1))


@pytest.mark.parametrize("nq,k", [(1, 64), (1, 512), (64, 512), (36, 1024), (160, 256)])
def test_a_nan_row_shows_however_the_query_is_split(csa, nq, k):
    N, H, c = 300, 64, 512
    kv, _ = _rows(csa, N, c, 64, 61)
    kv[7] = 255
    g = _gen(k)
    q = torch.randn(nq, H, c, generator=g).to(torch.bfloat16).to(DEV)
    idx = torch.randint(8, N, (nq, k), generator=g, dtype=torch.int32)
    idx[0, k - 2] = 7
    out, lse = csa.csa_sparse_mqa_fp4kv(q, kv, idx.to(DEV), seq_of_q=torch.zeros(nq, dtype=torch.int32, device=DEV))
    assert out[0].isnan().all() and lse[0].isnan().all()
    assert out[1:].isfinite().all() and lse[1:].isfinite().all()


def test_sparse_attention_odd_lists(csa):
    # indices past the cache, sequences out of range, logits far apart, a scale of one's own
    B, N, H, c, R, k = 2, 50, 64, 512, 64, 160
    kv, V = _rows(csa, B * N, c, R, 4, scale=3.0)
    kv, V = kv.reshape(B, N, -1), V.reshape(B, N, c)
    g = _gen(9)
    q = (30 * torch.randn(4, H, c, generator=g)).to(torch.bfloat16)
    idx = torch.randint(-3, N + 20, (4, k), generator=g, dtype=torch.int32)
    idx[0, 0], idx[0, 1] = 2 ** 31 - 1, -2 ** 31
    seq = torch.tensor([0, 1, 2, -1], dtype=torch.int32)
    out, lse = csa.csa_sparse_mqa_fp4kv(q.to(DEV), kv, idx.to(DEV), scale=0.01, seq_of_q=seq.to(DEV))
    ids = idx.numpy().copy()
    ids[(ids >= N) | (ids < 0)] = -1
    ids[2:] = -1
    check_attention(out, lse, q, V, ids, 0.01, None, np.array([0, 1, 0, 0]))
    assert (host(out)[2:] == 0).all() and np.isneginf(host(lse)[2:]).all()


def test_a_selected_nan_row_shows(csa):
    kv, _ = _rows(csa, 40, 512, 64, 5)
    kv[7] = 255
    q = torch.randn(2, 64, 512, generator=_gen(1)).to(torch.bfloat16).to(DEV)
    idx = torch.tensor([[1, 7, 3], [1, 2, 3]], dtype=torch.int32, device=DEV)
    out, lse = csa.csa_sparse_mqa_fp4kv(q, kv, idx, seq_of_q=torch.zeros(2, dtype=torch.int32, device=DEV))
    assert out[0].isnan().all() and lse[0].isnan().all()
    assert out[1].isfinite().all() and lse[1].isfinite().all()


# ---------------------------------------------------------------- attention over all visible entries
@pytest.mark.parametrize("N,H,c,R,lens", [
    (300, 64, 512, 64, [0, 1, 127, 128, 129, 300]), (2000, 64, 512, 64, [2000, 1999]), (70, 128, 512, 0, [70, 3, 0]),
    (1500, 40, 256, 32, [0, 1500, 1]), (40, 7, 128, 96, [40] * 12), (9000, 64, 384, 96, [8999])])
@pytest.mark.parametrize("with_sink", [False, True])
def test_dense_attention(csa, N, H, c, R, lens, with_sink):
    B = len(lens)
    kv, V = _rows(csa, B * N, c, R, 6)
    kv, V = kv.reshape(B, N, -1), V.reshape(B, N, c).copy()
    g = _gen(N)
    q = (2 * torch.randn(B, H, c, generator=g)).to(torch.bfloat16)
    sink = torch.randn(H, generator=g) if with_sink else None
    idx = np.full((B, N), -1, np.int32)
    for b, n in enumerate(lens):
        idx[b, :n] = np.arange(n)
        kv[b, n:] = 255                                   # rows behind the last visible entry: NaN
        V[b, n:] = 0
    pos = torch.tensor(lens, dtype=torch.int32) * 128 + 127
    pos[lens.index(max(lens))] = 2 ** 31 - 1              # past the cache: every entry, once its rows are real
    if max(lens) < N:
        pos[lens.index(max(lens))] = max(lens) * 128
    keep = kv.clone()
    out, lse = csa.hca_decode_fp4kv(q.to(DEV), kv, pos.to(DEV), 128, rope_dims=R,
                                    sink=None if sink is None else sink.to(DEV))
    check_attention(out, lse, q, V, idx, 1 / math.sqrt(c), None if sink is None else sink.double().numpy(),
                    np.arange(B))
    out2, lse2 = csa.hca_decode_fp4kv(q.to(DEV), kv, pos.to(DEV), 128, rope_dims=R,
                                      sink=None if sink is None else sink.to(DEV))
    assert torch.equal(out, out2) and torch.equal(lse, lse2) and torch.equal(kv, keep)


def test_dense_attention_many_queries_of_few_sequences(csa):
    B, N, H, c, R, nq = 2, 333, 16, 256, 64, 50
    kv, V = _rows(csa, B * N, c, R, 7)
    kv, V = kv.reshape(B, N, -1), V.reshape(B, N, c)
    g = _gen(70)
    q = torch.randn(nq, H, c, generator=g).to(torch.bfloat16)
    pos = torch.randint(-4, 4 * N + 40, (nq,), generator=g, dtype=torch.int32)
    seq = torch.randint(0, B, (nq,), generator=g, dtype=torch.int32)
    out, lse = csa.hca_dense_mqa_fp4kv(q.to(DEV), kv, pos.to(DEV), 4, seq_of_q=seq.to(DEV))
    idx = np.full((nq, N), -1, np.int32)
    for t in range(nq):
        n = min(N, max(0, int(pos[t])) // 4)
        idx[t, :n] = np.arange(n)
    check_attention(out, lse, q, V, idx, 1 / 16, None, seq.numpy())


def test_offsets_past_32_bits(csa):
    # a cache of 4.7 GB: the rows read lie behind the 2^32nd byte
    B, N, c, R, H, k = 3, 4_100_000, 512, 64, 64, 256
    kv = torch.zeros(B, N, 384, dtype=torch.uint8, device=DEV)
    rows, V = _rows(csa, 600, c, R, 8)
    kv[2, N - 600:] = rows
    q = (2 * torch.randn(1, H, c, generator=_gen(2))).to(torch.bfloat16)
    idx = torch.randperm(600, generator=_gen(3))[:k].to(torch.int32)[None]
    two = torch.full((1,), 2, dtype=torch.int32, device=DEV)
    out, lse = csa.csa_sparse_mqa_fp4kv(q.to(DEV), kv, (idx + (N - 600)).to(DEV), seq_of_q=two)
    check_attention(out, lse, q, V[None], idx.numpy(), c ** -0.5, None, np.array([0]))
    w = csa.csa_entry_weights_fp4kv(q.to(DEV), lse, kv, (idx + (N - 600)).to(DEV), seq_of_q=two)
    ref = oracle.entry_weights(host(q), host(lse), V[None], idx.numpy(), c ** -0.5, np.array([0]))
    check_weights(w, ref, _logit_slack(host(q), V[None], c ** -0.5))
    del kv


# ---------------------------------------------------------------- weights
@pytest.mark.parametrize("nq,B,N,H,c,R,k", [(1, 1, 5, 1, 128, 0, 3), (3, 3, 300, 64, 512, 64, 512),
                                            (2, 2, 150, 128, 512, 64, 129), (5, 2, 90, 24, 256, 32, 37)])
def test_weights_of_a_selection(csa, nq, B, N, H, c, R, k):
    kv, V = _rows(csa, B * N, c, R, 11)
    kv, V = kv.reshape(B, N, -1), V.reshape(B, N, c)
    g = _gen(k)
    q = (2 * torch.randn(nq, H, c, generator=g)).to(torch.bfloat16)
    idx = torch.randint(-N // 4, N, (nq, k), generator=g, dtype=torch.int32)
    if nq > 1:
        idx[1] = -1
    seq = None if B == nq else torch.arange(nq, dtype=torch.int32) % B
    dev = dict(seq_of_q=None if seq is None else seq.to(DEV), rope_dims=R)
    used = torch.zeros(B, N, dtype=torch.bool)
    for t in range(nq):
        used[t % B, idx[t][idx[t] >= 0].long()] = True
    kv[~used.to(DEV)] = 255
    V = np.where(used.numpy()[..., None], V, 0)
    _, lse = csa.csa_sparse_mqa_fp4kv(q.to(DEV), kv, idx.to(DEV), **dev)
    ref = oracle.entry_weights(host(q), host(lse), V, idx.numpy(), c ** -0.5, np.arange(nq) % B)
    dz = _logit_slack(host(q), V, c ** -0.5)
    w = csa.csa_entry_weights_fp4kv(q.to(DEV), lse, kv, idx.to(DEV), **dev)
    check_weights(w, ref, dz)
    if seq is None:
        start = torch.rand(B, N, generator=g)
        acc = start.to(DEV)
        csa.csa_entry_weights_fp4kv(q.to(DEV), lse, kv, idx.to(DEV), acc=acc, **dev)
        want = start.double().numpy()
        for t in range(nq):
            for i in np.flatnonzero(idx[t].numpy() >= 0):
                want[t, idx[t, i]] += host(w)[t, i]
        # a sum of up to k + 1 terms
        np.testing.assert_allclose(host(acc), want, rtol=(k + 1) * 2.0 ** -24, atol=0)
        other = start.to(DEV)
        csa.csa_entry_weights_fp4kv(q.to(DEV), lse, kv, idx.to(DEV), acc=other, **dev)
        assert torch.equal(acc, other)


@pytest.mark.parametrize("B,T,N,H,c,R", [(6, 1, 300, 64, 512, 64), (2, 3, 140, 128, 512, 0), (1, 17, 700, 40, 256, 32),
                                         (3, 2, 129, 1, 128, 96), (1, 4, 129, 65, 384, 0)])
def test_weights_of_every_entry(csa, B, T, N, H, c, R):
    kv, V = _rows(csa, B * N, c, R, 12)
    kv, V = kv.reshape(B, N, -1), V.reshape(B, N, c).copy()
    g = _gen(B + T)
    q = (2 * torch.randn(B, T, H, c, generator=g)).to(torch.bfloat16)
    lens = torch.randint(0, N + 1, (B, T), generator=g)
    lens[0, 0] = N
    if B > 2:
        lens[1], lens[2, 0] = 0, 1
    lse = torch.zeros(B, T, H)
    ref = np.zeros((B, N))
    for b in range(B):
        kv[b, int(lens[b].max()):] = 255
        V[b, int(lens[b].max()):] = 0
        for t in range(T):
            n = int(lens[b, t])
            idx = np.arange(n, dtype=np.int32)[None] if n else np.full((1, 1), -1, np.int32)
            _, l = oracle.sparse_mqa(host(q[b, t])[None], V[b][None], idx, c ** -0.5, seq=np.zeros(1))
            lse[b, t] = torch.from_numpy(l[0]).float()
            ref[b, :n] += oracle.entry_weights(host(q[b, t])[None], host(lse[b, t])[None], V[b][None], idx, c ** -0.5,
                                               np.zeros(1, int))[0][:n]
    dz = _logit_slack(host(q).reshape(B * T, H, c), V, c ** -0.5)
    pos = (lens * 4 + 3).int()
    args = (q.to(DEV), lse.to(DEV), kv, pos.to(DEV), 4)
    w = csa.hca_entry_weights_fp4kv(*args, rope_dims=R)
    check_weights(w, ref, dz)
    acc = torch.rand(B, N, generator=g).to(DEV)
    out = csa.hca_entry_weights_fp4kv(*args, acc=acc, rope_dims=R)
    assert torch.equal(out, acc + w)
    csa.hca_entry_weights_fp4kv(*args, acc=acc, rope_dims=R, out=acc)
    assert torch.equal(out, acc)
    if T == 1:
        flat = csa.hca_entry_weights_fp4kv(args[0][:, 0].contiguous(), args[1][:, 0].contiguous(), kv,
                                           args[3][:, 0].contiguous(), 4, rope_dims=R)
        assert torch.equal(flat, w)


# ---------------------------------------------------------------- the decode step, graphs, streams
def test_decode_selects_like_csa_decode(csa):
    B, N, H, c, R, HI, cI, k, m = 4, 1024, 64, 512, 64, 64, 128, 256, 4
    g = _gen(21)
    x = torch.randn(B, N, c, generator=g).to(torch.bfloat16)
    kv = csa.csa_quantize_kv_fp4(x.to(DEV))
    V = oracle.dequantize_kv_fp4(kv.cpu().numpy(), c, R)
    K = torch.randn(B, N, cI, generator=g).to(torch.bfloat16).to(DEV)
    qI = torch.randn(B, HI, cI, generator=g).to(torch.bfloat16).to(DEV)
    w = torch.softmax(torch.randn(B, HI, generator=g), -1).to(DEV)
    q = torch.randn(B, H, c, generator=g).to(torch.bfloat16)
    sink = torch.randn(H, generator=g)
    ctx = torch.tensor([N * m, 2 * m + 1, 0, 2000], dtype=torch.int32).to(DEV)
    out, lse, sel = csa.csa_decode_fp4kv(qI, w, K, q.to(DEV), kv, ctx, m, k, sink=sink.to(DEV), return_topk=True)
    _, _, want = csa.csa_decode(qI, w, K, q.to(DEV), x.to(DEV), ctx, m, k, return_topk=True)
    assert torch.equal(sel, want)
    check_attention(out, lse, q, V, sel.cpu().numpy(), c ** -0.5, sink.double().numpy(), np.arange(B))
    out2, _ = csa.csa_decode_fp4kv(qI, w, K, q.to(DEV), kv, ctx, m, k, sink=sink.to(DEV))
    assert torch.equal(out, out2)


def test_captured_step_replays(csa):
    B, N, H, c, k = 3, 700, 64, 512, 200
    kv, _ = _rows(csa, B * N, c, 64, 31)
    kv = kv.reshape(B, N, -1)
    g = _gen(5)
    q = torch.randn(B, H, c, generator=g).to(torch.bfloat16).to(DEV)
    idx = torch.randint(0, N, (B, k), generator=g, dtype=torch.int32).to(DEV)
    pos = torch.tensor([N, 5, 333], dtype=torch.int32, device=DEV)
    new = torch.randn(B, c, generator=g).to(torch.bfloat16).to(DEV)
    slot = torch.tensor([3, 0, -1], dtype=torch.int32, device=DEV)
    acc = torch.zeros(B, N, device=DEV)

    def step():
        csa.csa_append_kv_fp4(new, slot, kv)
        o1, l1 = csa.csa_sparse_mqa_fp4kv(q, kv, idx)
        o2, l2 = csa.hca_dense_mqa_fp4kv(q, kv, pos, 1)
        csa.csa_entry_weights_fp4kv(q, l1, kv, idx, acc=acc)
        csa.hca_entry_weights_fp4kv(q, l2, kv, pos, 1, acc=acc, out=acc)
        return o1, l1, o2, l2

    eager = [t.clone() for t in step()]
    first = acc.clone()
    acc.zero_()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step()
    for _ in range(2):
        acc.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(eager, outs)) and torch.equal(acc, first)
    q.mul_(0.5)
    acc.zero_()
    graph.replay()
    got = [t.clone() for t in outs]
    acc.zero_()
    assert all(torch.equal(a, b) for a, b in zip(got, step()))


def test_two_streams_at_once(csa):
    B, N, H, c, k = 2, 3000, 64, 512, 512
    kv, _ = _rows(csa, B * N, c, 64, 41)
    kv = kv.reshape(B, N, -1)
    g = _gen(6)
    q = [torch.randn(B, H, c, generator=g).to(torch.bfloat16).to(DEV) for _ in range(2)]
    idx = torch.randint(0, N, (B, k), generator=g, dtype=torch.int32).to(DEV)
    pos = torch.full((B,), N, dtype=torch.int32, device=DEV)
    want = [csa.csa_sparse_mqa_fp4kv(x, kv, idx)[0] for x in q] + [csa.hca_dense_mqa_fp4kv(x, kv, pos, 1)[0] for x in q]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = {}
    for rep in range(5):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                got[i] = csa.csa_sparse_mqa_fp4kv(q[i], kv, idx)[0]
                got[2 + i] = csa.hca_dense_mqa_fp4kv(q[i], kv, pos, 1)[0]
        torch.cuda.synchronize()
        assert all(torch.equal(got[i], want[i]) for i in range(4))


def test_binding_refusals(csa):
    kv = torch.zeros(2, 8, 384, dtype=torch.uint8, device=DEV)
    q = torch.zeros(2, 4, 512, dtype=torch.bfloat16, device=DEV)
    idx = torch.zeros(2, 3, dtype=torch.int32, device=DEV)
    for bad in (dict(q=q.float()), dict(idx=idx.long()), dict(kv=kv[..., :368]), dict(q=q[:, :, :256]),
                dict(idx=idx[:1]), dict(kv=kv.cpu()), dict(q=q.transpose(0, 1)), dict(sink=torch.zeros(3, device=DEV))):
        a = dict(q=q, kv=kv, idx=idx, sink=None)
        a.update(bad)
        with pytest.raises((ValueError, csa.CsaError)):
            csa.csa_sparse_mqa_fp4kv(a["q"], a["kv"], a["idx"], sink=a["sink"])
    with pytest.raises(csa.CsaError):
        csa.csa_sparse_mqa_fp4kv(q, kv, idx, out=q)
    with pytest.raises(ValueError):
        csa.csa_quantize_kv_fp4(q[..., ::2])
    with pytest.raises(ValueError):
        csa.hca_decode_fp4kv(q, kv[:1], torch.zeros(2, dtype=torch.int32, device=DEV), 4)
    torch.cuda.synchronize()


def test_empty_batches_and_caches(csa):
    z = lambda *shape, dt=torch.bfloat16: torch.zeros(shape, dtype=dt, device=DEV)
    i32, u8, f32 = torch.int32, torch.uint8, torch.float32
    assert csa.csa_quantize_kv_fp4(z(0, 512)).shape == (0, 384)
    assert csa.csa_dequantize_kv_fp4(z(0, 384, dt=u8), 512).shape == (0, 512)
    csa.csa_append_kv_fp4(z(0, 512), z(0, dt=i32), z(0, 9, 384, dt=u8))
    csa.csa_append_kv_fp4(z(2, 512), z(2, dt=i32), z(2, 0, 384, dt=u8))
    out, lse = csa.csa_sparse_mqa_fp4kv(z(0, 4, 512), z(0, 9, 384, dt=u8), z(0, 3, dt=i32))
    assert out.shape == (0, 4, 512) and lse.shape == (0, 4)
    assert csa.hca_decode_fp4kv(z(0, 4, 512), z(0, 9, 384, dt=u8), z(0, dt=i32), 4)[0].shape == (0, 4, 512)
    assert csa.csa_entry_weights_fp4kv(z(0, 4, 512), z(0, 4, dt=f32), z(0, 9, 384, dt=u8), z(0, 3, dt=i32)).shape == (0, 3)
    assert csa.hca_entry_weights_fp4kv(z(0, 4, 512), z(0, 4, dt=f32), z(0, 9, 384, dt=u8), z(0, dt=i32), 4).shape == (0, 9)
    # caches without rows: the sink logit, or nothing
    q, sink = torch.ones(2, 4, 512, dtype=torch.bfloat16, device=DEV), torch.tensor([0.5, -1.0, 2.0, 0.0], device=DEV)
    for call in (lambda s: csa.csa_sparse_mqa_fp4kv(q, z(2, 0, 384, dt=u8), z(2, 3, dt=i32), sink=s),
                 lambda s: csa.hca_decode_fp4kv(q, z(2, 0, 384, dt=u8), z(2, dt=i32) + 99, 4, sink=s)):
        out, lse = call(None)
        assert (out == 0).all() and lse.isneginf().all()
        out, lse = call(sink)
        # the logarithm of e^sink / 1: a logarithm and a product, each within 2^-22 of its value
        assert (out == 0).all() and ((lse - sink).abs() <= 2.0 ** -21 * (1 + sink.abs())).all()
    acc = torch.ones(2, 5, device=DEV)
    no_t = csa.hca_entry_weights_fp4kv(z(2, 0, 4, 512), z(2, 0, 4, dt=f32), z(2, 5, 384, dt=u8), z(2, 0, dt=i32), 4, acc=acc)
    assert torch.equal(no_t, acc)


def test_calls_stay_on_their_stream(csa):
    # inputs made on a side stream, the call on that stream, the result read on it: no other stream is touched
    side = torch.cuda.Stream()
    g = _gen(77)
    x = torch.randn(4, 600, 512, generator=g).to(torch.bfloat16)
    q = torch.randn(4, 64, 512, generator=g).to(torch.bfloat16)
    pos = torch.tensor([600, 1, 0, 599], dtype=torch.int32)
    want = csa.hca_decode_fp4kv(q.to(DEV), csa.csa_quantize_kv_fp4(x.to(DEV)), pos.to(DEV), 1)
    torch.cuda.synchronize()
    for _ in range(3):
        with torch.cuda.stream(side):
            torch.cuda._sleep(2_000_000)
            xs = x.pin_memory().to(DEV, non_blocking=True)
            kv = csa.csa_quantize_kv_fp4(xs)
            got = csa.hca_decode_fp4kv(q.to(DEV), kv, pos.to(DEV), 1)
            same = [torch.equal(a, b) for a, b in zip(got, want)]
        assert all(same)


def test_weights_of_a_long_prompt_add_up(csa):
    # 1500 queries of two sequences in one call, and in three with acc = out
    B, T, N, H, c, R = 2, 1500, 200, 8, 128, 32
    kv, V = _rows(csa, B * N, c, R, 90)
    kv, V = kv.reshape(B, N, -1), V.reshape(B, N, c)
    g = _gen(91)
    q = torch.randn(B, T, H, c, generator=g).to(torch.bfloat16)
    pos = torch.randint(0, 4 * N + 9, (B, T), generator=g, dtype=torch.int32)
    ref = np.zeros((B, N))
    lse = np.zeros((B, T, H), np.float32)
    for b in range(B):
        z = np.einsum("thc,nc->thn", host(q[b]), V[b]) * c ** -0.5
        seen = np.arange(N)[None] < np.minimum(N, pos[b].numpy() // 4)[:, None]
        z = np.where(seen[:, None], z, -np.inf)
        m = z.max(-1, keepdims=True)
        m = np.where(np.isfinite(m), m, 0)
        with np.errstate(divide="ignore"):
            lse[b] = (m[..., 0] + np.log(np.exp(z - m).sum(-1))).astype(np.float32)
        ok = np.isfinite(lse[b])
        ref[b] = np.exp(z - np.where(ok, lse[b], 0)[..., None])[ok].sum(0)
    dz = _logit_slack(host(q).reshape(B * T, H, c), V, c ** -0.5)
    args = (q.to(DEV), torch.from_numpy(lse).to(DEV), kv, pos.to(DEV), 4)
    w = csa.hca_entry_weights_fp4kv(*args, rope_dims=R)
    # T sums of 64 fp32 terms on top of the single query's bound
    lim = (math.expm1(dz) + 2.0 ** -18 + (T + H) * 2.0 ** -24) * ref + 1e-37
    assert (np.abs(host(w) - ref) <= lim).all()
    acc = torch.zeros(B, N, device=DEV)
    for a, b in ((0, 700), (700, 701), (701, T)):
        part = [x[:, a:b].contiguous() for x in (args[0], args[1])] + [kv, args[3][:, a:b].contiguous(), 4]
        csa.hca_entry_weights_fp4kv(*part, acc=acc, rope_dims=R, out=acc)
    assert (np.abs(host(acc) - ref) <= lim).all()

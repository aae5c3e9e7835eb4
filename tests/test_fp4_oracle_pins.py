"""Pins of the oracle's 4-bit entry format and eviction order (no GPU)."""
import numpy as np
import torch

import oracle


def _bf16(a):
    return torch.from_numpy(np.asarray(a, dtype=np.float64)).to(torch.bfloat16).double().numpy()


def test_row_size_and_layout_by_hand():
    assert oracle.fp4_row_bytes(512, 64) == 224 + 32 + 128
    assert oracle.fp4_row_bytes(128, 0) == 64 + 16
    x = np.zeros(128)
    # block 0: max 6 -> scale 1; channels 0..7 in the first word
    x[:8] = [6, -6, 0.5, 1, 1.5, 2, 3, -4]
    x[16] = 0.75                       # block 1: scale 1/8, code 7
    row = oracle.quantize_kv_fp4(x, 32)
    # nibbles 0..3: channels 0 2 4 6; 4..7: channels 1 3 5 7
    assert list(row[:4]) == [0x17, 0x53, 0x2F, 0xE4]
    assert row[48] == 8 * 31 and row[49] == 8 * 28 and row[48 + 6] == 127
    assert row[48 + 2] == 0            # an empty block: the smallest scale
    v = oracle.dequantize_kv_fp4(row, 128, 32)
    np.testing.assert_array_equal(v, x)


def test_ties_go_to_the_even_code_and_the_even_scale():
    x = np.zeros(128)
    x[:9] = [6, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, -5.0]
    v = oracle.dequantize_kv_fp4(oracle.quantize_kv_fp4(x, 0), 128, 0)
    np.testing.assert_array_equal(v[:9], [6, 0, 1, 1, 2, 2, 4, 4, -4])
    x[0] = 6 * (1 + 1 / 16)            # scale 1 + 1/16: between 1 and 1 + 1/8
    assert oracle.quantize_kv_fp4(x, 0)[64] % 8 == 0
    x[0] = 6 * (1 + 3 / 16)
    assert oracle.quantize_kv_fp4(x, 0)[64] % 8 == 2


def test_error_bound_and_range():
    g = torch.Generator().manual_seed(5)
    x = torch.randn(40, 256, generator=g) * torch.exp(20 * torch.randn(40, 1, generator=g))
    x = _bf16(x.double().numpy())
    v = oracle.dequantize_kv_fp4(oracle.quantize_kv_fp4(x, 64), 256, 64)
    np.testing.assert_array_equal(v[:, 192:], x[:, 192:])
    b = np.abs(x[:, :192]).reshape(40, 12, 16)
    # the scale is within 1/16 of max/6; the widest code gap (4 to 6) then
    # leaves half of 2 scales, and what saturates at most 1/16 of the max
    lim = b.max(-1, keepdims=True) / 6 * (1 + 1 / 16)
    assert (np.abs(v[:, :192] - x[:, :192]).reshape(40, 12, 16) <= lim).all()
    np.testing.assert_array_equal(_bf16(v), v)          # every value is a bf16 number
    for big in (3.3895e38, -3.3895e38, 1e-38, -1e-40):
        y = _bf16(np.full(128, big))
        u = oracle.dequantize_kv_fp4(oracle.quantize_kv_fp4(y, 0), 128, 0)
        assert np.isfinite(u).all() and (np.abs(u) <= 1.07 * np.abs(y)).all()
    y = np.zeros(128)
    y[3] = np.inf
    assert np.isnan(oracle.dequantize_kv_fp4(oracle.quantize_kv_fp4(y, 32), 128, 32)[:96]).all()


def test_weights_of_a_full_attention_sum_to_the_heads():
    g = torch.Generator().manual_seed(6)
    q, KV = torch.randn(2, 3, 128, generator=g), torch.randn(2, 9, 128, generator=g)
    idx = np.tile(np.arange(9, dtype=np.int32), (2, 1))
    idx[1, 4] = -1
    _, lse = oracle.sparse_mqa(q, KV, idx, 0.1, seq=np.arange(2))
    w = oracle.entry_weights(q, lse, KV, idx, 0.1, np.arange(2))
    np.testing.assert_allclose(w.sum(1), 3.0, rtol=1e-12)
    assert w[1, 4] == 0


def test_evict_plan_by_hand():
    acc = np.array([5.0, 1.0, np.nan, 4.0, 9.0, 1.0, 7.0, -0.0])
    moves, left = oracle.evict_plan(acc, 8, 4)
    assert moves == [(4, 1), (6, 2)] and left == 4      # kept: 9 7 5 4
    assert oracle.evict_plan(acc, 3, 4) == ([], 3)
    # equal weights: the lower index stays
    assert oracle.evict_plan(np.ones(6), 6, 3) == ([], 3)
    # a protected entry stays whatever its weight
    moves, _ = oracle.evict_plan(acc, 8, 2, pos=np.arange(8), protect_from=7)
    assert moves == [(4, 0), (7, 1)]

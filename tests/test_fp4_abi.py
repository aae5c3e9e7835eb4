"""Refusals of the 4-bit cache and eviction entry points (no GPU: every check
comes before the first launch), and the binding's own checks."""
import pytest
import torch

import compressed_sparse_attention_14_b200 as csa

L = csa._lib
F = 0x10000  # 16-byte aligned, never dereferenced: checks fail first
BAD, UNSUP, WS = csa.CSA_ERR_INVALID_ARG, csa.CSA_ERR_UNSUPPORTED, csa.CSA_ERR_WORKSPACE


def test_row_bytes():
    assert csa.csa_fp4_row_bytes(512, 64) == 384
    assert csa.csa_fp4_row_bytes(128, 0) == 80
    assert csa.csa_fp4_row_bytes(256, 32) == 112 + 16 + 64
    for c, R in ((96, 32), (640, 64), (512, 16), (512, 512), (128, -32), (0, 0)):
        assert L.csa_fp4_row_bytes(c, R) == 0
        with pytest.raises(csa.CsaError):
            csa.csa_fp4_row_bytes(c, R)


def test_storage_refusals():
    assert L.csa_quantize_kv_fp4(F, 4, 96, 32, F, None) == UNSUP
    assert L.csa_quantize_kv_fp4(F, 4, 512, 40, F, None) == UNSUP
    assert L.csa_quantize_kv_fp4(F, -1, 512, 64, F, None) == BAD
    assert L.csa_quantize_kv_fp4(None, 4, 512, 64, F, None) == BAD
    assert L.csa_quantize_kv_fp4(F, 4, 512, 64, F + 8, None) == BAD
    assert L.csa_quantize_kv_fp4(F, 1 << 40, 512, 64, F, None) == UNSUP
    assert L.csa_quantize_kv_fp4(None, 0, 512, 64, None, None) == 0
    assert L.csa_dequantize_kv_fp4(F, 4, 512, 64, None, None) == BAD
    assert L.csa_dequantize_kv_fp4(F, 4, 512, 480 + 32, F, None) == UNSUP
    assert L.csa_append_kv_fp4(F, None, 4, 512, 64, F, 8, None) == BAD
    assert L.csa_append_kv_fp4(F, F, -4, 512, 64, F, 8, None) == BAD
    assert L.csa_append_kv_fp4(F, F, 4, 512, 64, F, 1 << 30, None) == UNSUP


def _sparse(nq=4, n_seq=4, H=8, c=128, R=32, Nmax=16, k=4, q=F, kv=F, idx=F, seq=None, out=F, ws=None, nb=0):
    return L.csa_sparse_mqa_fp4kv(q, kv, idx, seq, nq, n_seq, H, c, R, Nmax, k, 0.0, None, out, None, ws, nb, None)


def _dense(nq=4, n_seq=4, H=8, c=128, R=32, Nmax=16, mp=4, q=F, kv=F, pos=F, out=F):
    return L.hca_dense_mqa_fp4kv(q, kv, pos, None, nq, n_seq, H, c, R, Nmax, mp, 0.0, None, out, None, F * 16, 1 << 40,
                                 None)


def test_attention_refusals():
    assert _sparse(H=0) == UNSUP and _sparse(H=129) == UNSUP
    assert _sparse(c=192) == UNSUP and _sparse(R=48) == UNSUP
    assert _sparse(k=0) == UNSUP and _sparse(k=2049) == UNSUP
    assert _sparse(nq=70000, n_seq=70000) == UNSUP
    assert _sparse(nq=-1) == BAD and _sparse(Nmax=-1) == BAD and _sparse(n_seq=0) == BAD
    assert _sparse(n_seq=3) == BAD and b"seq_of_q" in L.csa_last_error()
    assert _sparse(n_seq=1 << 16, Nmax=1 << 16) == UNSUP
    for name in ("q", "kv", "idx", "out"):
        assert _sparse(**{name: None}) == BAD and _sparse(**{name: F + 4}) == BAD
    assert _sparse(out=F) == BAD and b"overlap" in L.csa_last_error()      # out is q
    assert _sparse(nq=0) == 0
    assert _dense(mp=0) == BAD and _dense(pos=None) == BAD and _dense(nq=-2) == BAD
    need = L.csa_decode_fp4kv_workspace_size(2, 1024, 8, 128, 4, 64, 16)
    assert need > 0
    args = (F, F, F, F, F, F, 2, 1024, 4, 8, 128, 32, 4, 64, 16, 0.0, None, F * 2, None, None)
    assert L.csa_decode_fp4kv(*args, None, 0, None) == WS
    assert L.csa_decode_fp4kv(*args, F * 16, need - 1, None) == WS
    assert L.csa_decode_fp4kv(*args, F * 16 + 16, need, None) == WS
    assert L.csa_decode_fp4kv(F, F, F, F, F, F, 2, 1024, 0, 8, 128, 32, 4, 64, 16, 0.0, None, F, None, None, F * 16,
                              need, None) == BAD


def test_weight_refusals():
    def sp(seq=None, w=F, acc=None, lse=F, k=4):
        return L.csa_entry_weights_fp4kv(F, lse, F, F, seq, 4, 4, 8, 128, 32, 16, k, 0.0, w, acc, None)
    assert sp(seq=F, acc=F) == BAD and b"one query per sequence" in L.csa_last_error()
    assert sp(w=None) == BAD and sp(lse=None) == BAD and sp(k=0) == UNSUP

    def de(B=4, T=1, mp=4, out=F):
        return L.hca_entry_weights_fp4kv(F, F, F, F, B, T, 8, 128, 32, 16, mp, 0.0, None, out, None)
    assert de(T=-1) == BAD and de(mp=0) == BAD and de(out=None) == BAD and de(B=-1) == BAD
    assert de(B=60000, T=60000) == UNSUP
    assert de(B=0) == 0


def test_weights_of_more_queries_than_a_call_takes():
    def de(T):
        return L.hca_entry_weights_fp4kv(F, F, F, F, 1, T, 8, 128, 32, 16, 4, 0.0, None, None, None)
    assert de((1 << 18) + 1) == UNSUP and b"2^18" in L.csa_last_error()
    assert de(1 << 18) == BAD                                              # (out is missing)


def test_eviction_refusals():
    def plan(B=2, N=16, keep=8, pos=None, prot=None, pos_out=None, acc=F, acc_out=F, src=F):
        return L.csa_evict_plan(acc, F, pos, prot, B, N, keep, src, F, F, F, acc_out, pos_out, F * 16, 1 << 30, None)
    assert plan(keep=-1) == BAD and plan(keep=17) == BAD and plan(N=-1, keep=0) == BAD
    assert plan(prot=F) == BAD and plan(pos=F) == BAD and plan(pos_out=F) == BAD
    assert plan(acc=None) == BAD and plan(acc_out=F + 4) == BAD and plan(src=None) == BAD
    assert plan(B=70000) == UNSUP and plan(N=1 << 32, keep=4) == UNSUP
    assert plan(B=0) == 0

    def rows(rb=16, M=8, cache=F):
        return L.csa_evict_rows(cache, rb, 2, 16, F, F, F, M, None)
    assert rows(rb=24) == BAD and rows(rb=0) == BAD and rows(M=17) == BAD and rows(M=-1) == BAD
    assert rows(cache=None) == BAD and rows(M=0) == 0

    def slot(m=4, cap=8, recent=0, pos=None, acc=F):
        return L.csa_evict_slot(acc, F, pos, F, 2, 16, m, cap, recent, F, None)
    assert slot(m=0) == BAD and slot(cap=0) == BAD and slot(cap=17) == BAD and slot(recent=-1) == BAD
    assert slot(recent=2) == BAD and slot(acc=None) == BAD


def test_sizes_of_empty_calls():
    assert L.csa_sparse_mqa_fp4kv_workspace_size(0, 64, 512, 512) == 0
    assert L.csa_sparse_mqa_fp4kv_workspace_size(-1, 64, 512, 512) == 0
    assert L.csa_evict_plan_workspace_size(4, 16, 17) == 0


def test_binding_wants_cuda_tensors():
    x = torch.zeros(2, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        csa.csa_quantize_kv_fp4(x, rope_dims=32)
    with pytest.raises(ValueError, match="CUDA"):
        csa.csa_evict_plan(torch.zeros(2, 8), torch.zeros(2, dtype=torch.int32), 4)

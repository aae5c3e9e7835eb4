"""Measured cases of the 4-bit KV cache operators.

Operators: storing cache entries in 4 bits (and reading them back), shared-KV
attention over such a cache (selected entries, every visible entry), the
attention weight each entry received, and eviction by accumulated weight.

The 4-bit entry (c channels, the last R of them rotary and kept bf16; Q = c - R):

  bytes [0, Q/2)          codes, e2m1 (sign, 2 exponent bits, 1 mantissa bit:
                          0 .5 1 1.5 2 3 4 6); in each group of 8 channels the
                          4-byte word holds channel 2j in nibble j and channel
                          2j+1 in nibble j+4
  bytes [Q/2, Q/2+Q/16)   one scale byte s per 16 channels
  byte  Q/2+Q/16          row exponent E; zero padding to a multiple of 16
  then                    the R rotary channels, bf16

  value = e2m1 * (1 + (s mod 8)/8) * 2^(floor(s/8) - 31 + E - 127)

Writing it: a block's scale is max|x|/6 rounded to 4 significant bits (ties to
even), E the largest block exponent; a code is the e2m1 value nearest x / scale
(ties to the even code, saturating at 6).

`own = False` runs plain torch operations; `own = True` the library's calls.
"""
import math

import torch

own = False

DEV = "cuda"
_E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # one decode step's closed entries of a batch of 64, stored
        dict(name="quant_step", op="quant", rows=64, c=512, R=64),
        # one sequence's compressed cache (131072 tokens / 4) stored at once
        dict(name="quant_cache", op="quant", rows=32768, c=512, R=64),
        # one user, one decode step over 512 selected entries
        dict(name="sparse_one", op="sparse", nq=1, B=1, Nmax=32768, H=64, c=512, R=64, k=512, start=131072, sink=True),
        # the Flash decode batch
        dict(name="sparse_decode", op="sparse", nq=64, B=64, Nmax=32768, H=64, c=512, R=64, k=512, start=131072,
             sink=True),
        # 128 heads over 1024 selected entries (the Pro decode shape)
        dict(name="sparse_wide", op="sparse", nq=32, B=32, Nmax=65536, H=128, c=512, R=64, k=1024, start=262144,
             sink=False),
        # a prefill chunk from the start of a sequence: the first queries see
        # fewer than k entries, the very first none
        dict(name="sparse_prefill", op="sparse", nq=3001, B=1, Nmax=4099, H=64, c=512, R=64, k=512, start=0, sink=True),
        # a few users of a smaller model, one of them with no entry, one with one
        dict(name="dense_ragged", op="dense", B=3, Nmax=8193, H=40, c=256, R=32, sink=False),
        # the HCA decode batch
        dict(name="dense_decode", op="dense", B=16, Nmax=8192, H=64, c=512, R=64, sink=True),
        # attention weight received in that step
        dict(name="weights_dense", op="wdense", B=16, T=1, Nmax=8192, H=64, c=512, R=64),
        # and by the selected entries of the Flash decode batch
        dict(name="weights_sparse", op="wsparse", nq=64, B=64, Nmax=32768, H=64, c=512, R=64, k=512, start=131072),
        # a batch of caches brought down to half its entries
        dict(name="evict_half", op="evict", B=16, Nmax=8192, keep=4096, rb=384, protect=128),
        # long caches of odd length cut to a small budget
        dict(name="evict_long", op="evict", B=3, Nmax=50021, keep=4001, rb=384, protect=0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["quant", "sparse", "sparse", "dense", "dense", "wdense", "wsparse", "evict"])
    c = rng.choice([128, 256, 384, 512, 512])
    R = rng.choice([0, 32, 64, 64])
    H = rng.choice([1, rng.randint(2, 63), 64, rng.randint(65, 127), 128])
    if op == "quant":
        return dict(op=op, rows=_log(rng, 1, 32768), c=c, R=R)
    if op == "evict":
        B = _log(rng, 1, 64)
        n = _log(rng, 2, min(65536, 262144 // B))
        return dict(op=op, B=B, Nmax=n, keep=_log(rng, 1, n), rb=rng.choice([160, 256, 384]),
                    protect=rng.choice([0, 0, rng.randint(1, n)]))
    if op in ("dense", "wdense"):
        B = _log(rng, 1, 32)
        case = dict(op=op, B=B, Nmax=_log(rng, 2, min(32768, 131072 // B)), H=H, c=c, R=R)
        if op == "dense":
            case["sink"] = rng.random() < 0.5
        else:
            case["T"] = rng.choice([1, 1, rng.randint(2, 16)])
        return case
    # (weights over a single entry would be the number of heads whatever the inputs)
    k = _log(rng, 1 if op == "sparse" else 2, 2048)
    if op == "sparse" and rng.random() < 0.3:
        nq = _log(rng, 2, max(2, min(2048, 1048576 // k)))
        n = _log(rng, 1, 8192)
        return dict(op=op, nq=nq, B=1, Nmax=n, H=min(H, 64), c=c, R=R, k=k, start=rng.randint(3, 4 * n),
                    sink=rng.random() < 0.5)
    B = _log(rng, 1, max(1, min(64, 65536 // k)))
    n = _log(rng, 2, 32768)
    case = dict(op=op, nq=B, B=B, Nmax=n, H=H, c=c, R=R, k=k, start=rng.randint(8, 4 * n + 8))
    if op == "sparse":
        case["sink"] = rng.random() < 0.5
    return case


def row_bytes(c, R):
    return (c - R) // 2 + ((c - R) // 16 + 1 + 15) // 16 * 16 + 2 * R


def _lens(case):
    """Visible entries of each sequence of a dense case: none, one, the rest spread up to a full cache."""
    B, n = case["B"], case["Nmax"]
    if B < 3:
        return [n] * B
    return [0, 1] + [n - (i * n) // (2 * (B - 2)) for i in range(B - 2)] if n < 8192 or B < 8 else \
        [n - (i * n) // (2 * B) for i in range(B)]


def _seen(case):
    """Visible entries of each query of a sparse case (blocks of 4 tokens)."""
    one = case["B"] == 1 and case["nq"] > 1
    return [min(case["Nmax"], (case["start"] + (t if one else 0)) // 4) for t in range(case["nq"])]


def work(case):
    op = case["op"]
    if op == "quant":
        n, c = case["rows"], case["c"]
        # the entry in bf16 read, the 4-bit row written, its values written
        return dict(bytes=n * (2 * c + row_bytes(c, case["R"]) + 2 * c), flops=4 * n * c)
    if op == "evict":
        B, n, keep = case["B"], case["Nmax"], case["keep"]
        moves = keep * (n - keep) // n                   # expected rows that move
        return dict(bytes=B * (n * 16 + moves * (2 * case["rb"] + 8)), flops=B * n)
    H, c, rb = case["H"], case["c"], row_bytes(case["c"], case["R"])
    if op in ("dense", "wdense"):
        e = sum(_lens(case))
        T = case.get("T", 1)
        if op == "dense":
            return dict(bytes=e * rb + case["B"] * H * (4 * c + 4), flops=4 * e * H * c)
        return dict(bytes=e * rb + case["B"] * (T * H * (2 * c + 4) + case["Nmax"] * 8), flops=2 * e * T * H * c)
    e = sum(min(v, case["k"]) for v in _seen(case))
    rows = min(e, max(_seen(case))) if case["B"] == 1 else e      # one sequence's rows are shared
    if op == "sparse":
        return dict(bytes=rows * rb + case["nq"] * (H * (4 * c + 4) + 4 * case["k"]), flops=4 * e * H * c)
    return dict(bytes=rows * rb + case["nq"] * (H * (2 * c + 4) + 8 * case["k"]), flops=2 * e * H * c)


# ------------------------------------------------------------------ plain forms
def _quantise(x, R):
    """x [n, c] bf16 -> codes [n, Q] (0..15), scale bytes [n, Q/16], row exponents [n] (int64 all)."""
    n, c = x.shape
    Q = c - R
    v = x[:, :Q].double().reshape(n, Q // 16, 16)
    a = v.abs().amax(-1)
    f, e = torch.frexp(a / 6)                            # f in [1/2, 1)
    e = e.long() - 1
    m = torch.round((2 * f - 1) * 8).long()
    e, m = e + (m == 8).long(), torch.where(m == 8, 0, m)
    low = (a == 0) | (e < -94)
    e, m = torch.where(low, -94, e), torch.where(low, 0, m)
    high = (e * 8 + m) > 125 * 8 + 2
    e, m = torch.where(high, 125, e), torch.where(high, 2, m)
    er = e.amax(-1)
    s = torch.clamp_min(8 * (e - er[:, None] + 31) + m, 0)
    s = torch.where(e - er[:, None] < -31, 0, s)
    S = _scale(s, er[:, None] + 127)
    r = v.abs()
    code = torch.zeros_like(v, dtype=torch.long)
    for mid, even in ((0.25, 0), (0.75, 1), (1.25, 0), (1.75, 1), (2.5, 0), (3.5, 1), (5.0, 0)):
        b = (S * mid)[..., None]
        code += (r >= b) if even else (r > b)
    code += 8 * torch.signbit(v).long()
    return code.reshape(n, Q), s, er + 127


def _scale(s, E):
    """The scale a byte stands for, in 64 bits (assembled from its bits: powers of 2 by pow() may be an ulp off)."""
    return (((s >> 3) - 31 + E - 127 + 1023 << 52) | ((s & 7) << 49)).view(torch.float64)


def _pack(x, R):
    """x [n, c] bf16 -> the 4-bit rows [n, row_bytes] uint8."""
    n, c = x.shape
    Q = c - R
    code, s, E = _quantise(x, R)
    g = code.reshape(n, Q // 8, 4, 2)
    g = torch.cat((g[..., 0], g[..., 1]), -1)            # nibbles 0..7: the even channels, then the odd ones
    out = torch.zeros(n, row_bytes(c, R), dtype=torch.uint8, device=x.device)
    out[:, :Q // 2] = (g[..., 0::2] + 16 * g[..., 1::2]).reshape(n, Q // 2).to(torch.uint8)
    out[:, Q // 2:Q // 2 + Q // 16] = s.to(torch.uint8)
    out[:, Q // 2 + Q // 16] = E.to(torch.uint8)
    if R:
        out[:, -2 * R:] = x[:, Q:].contiguous().view(torch.uint8)
    return out


def _unpack(rows, c, R):
    """4-bit rows [..., row_bytes] -> their values [..., c] in 32 bits (exact)."""
    lead = rows.shape[:-1]
    rows = rows.reshape(-1, rows.shape[-1])
    n, Q = rows.shape[0], c - R
    b = rows[:, :Q // 2].int().reshape(n, Q // 8, 4)
    g = torch.stack((b & 15, b >> 4), -1).reshape(n, Q // 8, 2, 4)
    code = g.transpose(-1, -2).reshape(n, Q)
    s = rows[:, Q // 2:Q // 2 + Q // 16].long()
    E = rows[:, Q // 2 + Q // 16].long()
    S = _scale(s, E[:, None]).float()
    tab = torch.tensor(_E2M1 + tuple(-v for v in _E2M1), device=rows.device)
    v = (tab[code].reshape(n, Q // 16, 16) * S[..., None]).reshape(n, Q)
    if R:
        v = torch.cat((v, rows[:, -2 * R:].contiguous().view(torch.bfloat16).float()), -1)
    return v.reshape(*lead, c)


def _softmax_out(z, V, sink):
    """z [n, H, k] logits (-inf where masked), V [n, k, c], sink [H] or None -> out bf16, lse."""
    m = z.amax(-1, keepdim=True) if z.shape[-1] else torch.full(z.shape[:-1] + (1,), -math.inf, device=z.device)
    if sink is not None:
        m = torch.maximum(m, sink[:, None])
    ref = torch.where(torch.isinf(m), 0.0, m)
    p = torch.exp(z - ref)
    L = p.sum(-1, keepdim=True)
    if sink is not None:
        L = L + torch.exp(sink[:, None] - ref)
    out = torch.bmm(p, V) / torch.where(L == 0, 1.0, L)
    return out.to(torch.bfloat16), (ref + torch.log(L)).squeeze(-1)


def _sparse_logits(s, t0, t1):
    case = s["case"]
    idx = s["idx"][t0:t1].long()
    ok = idx >= 0
    seq = torch.zeros_like(idx[:, 0]) if s["seq"] is not None else torch.arange(t0, t1, device=DEV)
    V = _unpack(s["kv"][seq[:, None], idx.clamp_min(0)], case["c"], case["R"])
    z = torch.bmm(s["q"][t0:t1].float(), V.transpose(1, 2)) / math.sqrt(case["c"])
    return z.masked_fill(~ok[:, None, :], -math.inf), V, ok


def _chunks(case):
    step = max(1, (1 << 27) // (case["k"] * case["c"]))
    return [(t, min(case["nq"], t + step)) for t in range(0, case["nq"], step)]


def _run_plain(s):
    case = s["case"]
    op = case["op"]
    if op == "quant":
        return _unpack(_pack(s["x"], case["R"]), case["c"], case["R"]).to(torch.bfloat16)
    if op == "sparse":
        parts = []
        for t0, t1 in _chunks(case):
            z, V, _ = _sparse_logits(s, t0, t1)
            parts.append(_softmax_out(z, V, s["sink"]))
        return torch.cat([p[0] for p in parts]), torch.cat([p[1] for p in parts])
    if op == "wsparse":
        parts = []
        for t0, t1 in _chunks(case):
            z, _, ok = _sparse_logits(s, t0, t1)
            lse = s["lse"][t0:t1, :, None]
            parts.append(torch.exp(z - torch.where(torch.isinf(lse), 0.0, lse)).sum(1))
        return torch.cat(parts)
    if op == "evict":
        return _evict_plain(s)
    V = _unpack(s["kv"], case["c"], case["R"])
    vis = torch.arange(case["Nmax"], device=DEV) < (s["pos"] // 128).reshape(case["B"], -1, 1)
    if op == "dense":
        z = torch.bmm(s["q"].float(), V.transpose(1, 2)) / math.sqrt(case["c"])
        return _softmax_out(z.masked_fill(~vis, -math.inf), V, s["sink"])
    B, T, H, c = s["q"].shape
    z = torch.bmm(s["q"].float().reshape(B, T * H, c), V.transpose(1, 2)) / math.sqrt(c)
    lse = s["lse"].reshape(B, T * H, 1)
    p = torch.exp(z - torch.where(torch.isinf(lse), 0.0, lse)).reshape(B, T, H, -1)
    return s["acc"] + (p * vis[:, :, None, :]).sum((1, 2))


def _evict_plain(s):
    case, acc, pos, cache = s["case"], s["acc"], s["entry_pos"], s["cache"]
    B, N, keep = case["B"], case["Nmax"], case["keep"]
    col = torch.arange(N, device=DEV)
    n = s["n_ent"].long()
    live = col < n[:, None]
    w = torch.where(live, acc, -math.inf)
    order = torch.sort(w, dim=1, descending=True, stable=True).indices
    prot = (pos >= s["protect_from"][:, None]) & live
    for key in (prot, live):                             # later keys weigh more
        by = torch.sort(torch.gather(key, 1, order).int(), dim=1, descending=True, stable=True).indices
        order = torch.gather(order, 1, by)
    kept = torch.zeros(B, N, dtype=torch.bool, device=DEV)
    kept.scatter_(1, order[:, :keep], True)
    kept &= live
    cut = (n > keep)[:, None]
    hole = (col < keep) & ~kept & cut
    mover = (col >= keep) & kept & cut
    M = min(keep, N - keep)
    # the rows in order first, the rest (N) after them
    src = torch.sort(torch.where(mover, col, N), dim=1).values[:, :M]
    dst = torch.sort(torch.where(hole, col, N), dim=1).values[:, :M]
    src, dst = torch.where(src == N, -1, src), torch.where(dst == N, -1, dst)
    moves = hole.sum(1)
    n_out = torch.minimum(n, torch.full_like(n, keep))
    slot = torch.arange(B, device=DEV)[:, None].expand(B, M)[src >= 0]
    a, b = src[src >= 0], dst[src >= 0]
    acc_out, pos_out = acc.clone(), pos.clone()
    acc_out[slot, b], pos_out[slot, b] = acc[slot, a], pos[slot, a]
    gone = col >= n_out[:, None]
    acc_out[gone], pos_out[gone] = 0.0, -1
    cache[slot, b] = cache[slot, a]
    return src.int(), dst.int(), moves.int(), n_out.int(), acc_out, pos_out, cache


# ------------------------------------------------------------------ the library's calls
def _run_own(s):
    import compressed_sparse_attention_14_b200 as csa
    case = s["case"]
    op = case["op"]
    if op == "quant":
        return csa.csa_dequantize_kv_fp4(csa.csa_quantize_kv_fp4(s["x"], rope_dims=case["R"]), case["c"],
                                         rope_dims=case["R"])
    if op == "sparse":
        return csa.csa_sparse_mqa_fp4kv(s["q"], s["kv"], s["idx"], rope_dims=case["R"], sink=s["sink"],
                                        seq_of_q=s["seq"], ws=s["ws"])
    if op == "dense":
        return csa.hca_dense_mqa_fp4kv(s["q"], s["kv"], s["pos"], 128, rope_dims=case["R"], sink=s["sink"], ws=s["ws"])
    if op == "wsparse":
        return csa.csa_entry_weights_fp4kv(s["q"], s["lse"], s["kv"], s["idx"], rope_dims=case["R"], seq_of_q=s["seq"])
    if op == "wdense":
        return csa.hca_entry_weights_fp4kv(s["q"], s["lse"], s["kv"], s["pos"], 128, rope_dims=case["R"], acc=s["acc"])
    src, dst, moves, n_out, acc_out, pos_out = csa.csa_evict_plan(s["acc"], s["n_ent"], case["keep"],
                                                                  entry_pos=s["entry_pos"],
                                                                  protect_from=s["protect_from"], ws=s["ws"])
    csa.csa_evict_rows(s["cache"], src, dst, moves)
    return src, dst, moves, n_out, acc_out, pos_out, s["cache"]


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ------------------------------------------------------------------ inputs
def _entries(g, n, c):
    """Cache entries: normalised rows of slightly different size, a few channels larger than the rest."""
    x = torch.randn(n, c, generator=g, device=DEV)
    x *= torch.exp(0.3 * torch.randn(n, 1, generator=g, device=DEV))
    x[:, ::37] *= 3
    return x.to(torch.bfloat16)


def _cache(g, n, c, R):
    """n 4-bit rows, stored in pieces (the plain form's temporaries are large)."""
    out = torch.empty(n, row_bytes(c, R), dtype=torch.uint8, device=DEV)
    # entries repeat every 16384 rows, their order shuffled: rows of a long
    # cache need not all be different, and making them all would take longer
    # than the measurement
    base = _pack(_entries(g, min(n, 16384), c), R)
    for i in range(0, n, 16384):
        k = min(16384, n - i)
        out[i:i + k] = base[torch.randperm(base.shape[0], generator=g, device=DEV)[:k]]
    return out


def _workspace(s):
    """The scratch a program keeps for its calls."""
    if not own:
        return None
    import compressed_sparse_attention_14_b200 as csa
    case = s["case"]
    if case["op"] == "evict":
        nb = csa.workspace_size("csa_evict_plan", case["B"], case["Nmax"], case["keep"])
    elif case["op"] == "sparse":
        nb = csa.workspace_size("csa_sparse_mqa_fp4kv", case["nq"], case["H"], case["c"], case["k"])
    else:
        nb = csa.workspace_size("hca_dense_mqa_fp4kv", case["B"], case["H"], case["c"], case["Nmax"])
    return torch.empty(nb, dtype=torch.uint8, device=DEV) if nb else None


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    op = case["op"]
    s = dict(case=case)
    if op == "quant":
        s["x"] = _entries(g, case["rows"], case["c"])
        return s
    if op == "evict":
        B, N = case["B"], case["Nmax"]
        # few entries hold most of the weight, many hold none at all
        w = torch.exp(2 * torch.randn(B, N, generator=g, device=DEV) - 4)
        w[torch.rand(B, N, generator=g, device=DEV) < 0.2] = 0.0
        s["acc"] = w
        s["n_ent"] = torch.full((B,), N, dtype=torch.int32, device=DEV)
        s["entry_pos"] = torch.arange(N, dtype=torch.int32, device=DEV).repeat(B, 1)
        s["protect_from"] = torch.full((B,), N - case["protect"], dtype=torch.int32, device=DEV)
        s["cache"] = torch.randint(0, 256, (B, N, case["rb"]), generator=g, device=DEV, dtype=torch.uint8)
        s["ws"] = _workspace(s)
        return s
    B, N, H, c, R = case["B"], case["Nmax"], case["H"], case["c"], case["R"]
    s["kv"] = _cache(g, B * N, c, R).reshape(B, N, -1)
    if op in ("sparse", "wsparse"):
        nq, k = case["nq"], case["k"]
        s["q"] = (2 * torch.randn(nq, H, c, generator=g, device=DEV)).to(torch.bfloat16)
        seen = torch.tensor(_seen(case), device=DEV)
        # distinct entries of each query: k steps of a stride prime to the
        # number it sees, from a random start
        idx = torch.full((nq, k), -1, dtype=torch.int32, device=DEV)
        first = (torch.rand(nq, generator=g, device=DEV) * seen).long()
        stride = torch.tensor([next((p for p in (997, 991, 983) if v % p), 1) for v in _seen(case)], device=DEV)
        j = torch.arange(k, device=DEV)
        v = (first[:, None] + j * stride[:, None]) % seen.clamp_min(1)[:, None]
        idx = torch.where(j < torch.clamp_max(seen, k)[:, None], v, -1).int()
        s["idx"] = idx.contiguous()
        s["seq"] = torch.zeros(nq, dtype=torch.int32, device=DEV) if B == 1 and nq > 1 else None
        if op == "wsparse":
            s["lse"] = torch.cat([torch.logsumexp(_sparse_logits(s, a, b)[0], -1) for a, b in _chunks(case)])
    else:
        T = case.get("T", 1)
        shape = (B, H, c) if op == "dense" else (B, T, H, c)
        s["q"] = (2 * torch.randn(*shape, generator=g, device=DEV)).to(torch.bfloat16)
        lens = torch.tensor(_lens(case), dtype=torch.int32, device=DEV)
        s["pos"] = lens * 128 if op == "dense" else (lens * 128)[:, None].repeat(1, T).contiguous()
        if op == "wdense":
            s["acc"] = torch.rand(B, N, generator=g, device=DEV)
            V = _unpack(s["kv"], c, R)
            z = torch.bmm(s["q"].float().reshape(B, T * H, c), V.transpose(1, 2)) / math.sqrt(c)
            z.masked_fill_(~(torch.arange(N, device=DEV) < lens[:, None, None]), -math.inf)
            s["lse"] = torch.logsumexp(z, -1).reshape(B, T, H)
            del V, z
    s["sink"] = torch.randn(H, generator=g, device=DEV) if case.get("sink") else None
    if op in ("sparse", "dense"):
        s["ws"] = _workspace(s)
    return s


# ------------------------------------------------------------------ the definition in 64 bits
def _pow2(e):
    """2^e for whole e, exactly."""
    return (e.long() + 1023 << 52).view(torch.float64)


def _values64(rows, c, R):
    """Each byte of a 4-bit row taken apart channel by channel."""
    Q = c - R
    d = torch.arange(Q, device=rows.device)
    nib = (d % 8) // 2 + 4 * (d % 2)
    byte = rows[..., 4 * (d // 8) + nib // 2]
    code = torch.where(nib % 2 == 1, byte // 16, byte % 16)
    s = rows[..., Q // 2 + d // 16].double()
    E = rows[..., Q // 2 + Q // 16].double()[..., None]
    ex, man = torch.floor((code % 8).double() / 2), code.double() % 2
    mag = torch.where(ex == 0, man * 0.5, (1 + man / 2) * _pow2(ex - 1))
    v = torch.where(code >= 8, -mag, mag) * (1 + (s % 8) / 8) * _pow2(torch.floor(s / 8) + E - 158)
    if R:
        v = torch.cat((v, rows[..., -2 * R:].contiguous().view(torch.bfloat16).double()), -1)
    return v


def _exact_quant(x, R):
    Q = x.shape[1] - R
    v = x[:, :Q].double().reshape(x.shape[0], -1, 16)
    t = v.abs().amax(-1) / 6
    t = t.clamp(2.0 ** -94, 1.25 * 2.0 ** 125)
    e = torch.floor(torch.log2(t))
    e = torch.where(_pow2(e) > t, e - 1, torch.where(_pow2(e + 1) <= t, e + 1, e))
    steps = 1 + torch.arange(9, device=x.device, dtype=torch.float64) / 8
    # the nearest step; of two as near, the even one (odd steps a hair further)
    far = (t / _pow2(e))[..., None].sub(steps).abs() + 1e-9 * (torch.arange(9, device=x.device) % 2)
    S = steps[far.argmin(-1)] * _pow2(e)
    top = (torch.frexp(S).exponent - 1).amax(-1, keepdim=True)
    S = torch.maximum(S, _pow2(top - 31))
    grid = torch.tensor(_E2M1, device=x.device, dtype=torch.float64)
    best = None
    for i in range(8):
        gap = (v.abs() / S[..., None] - grid[i]).abs() + 1e-9 * (i % 2)
        if best is None:
            best, out = gap, torch.full_like(v, grid[i].item())
        else:
            out = torch.where(gap < best, grid[i], out)
            best = torch.minimum(best, gap)
    out = (out * S[..., None] * torch.where(v < 0, -1.0, 1.0)).reshape(x.shape[0], Q)
    return torch.cat((out, x[:, Q:].double()), -1)


def exact(case, seed):
    op = case["op"]
    s = prepare(case, seed)
    if op == "quant":
        return _exact_quant(s["x"], case["R"])
    if op == "evict":
        return None
    c, R, scale = case["c"], case["R"], case["c"] ** -0.5
    sink = None if s.get("sink") is None else s["sink"].double()
    outs, extra = [], []
    sparse = op in ("sparse", "wsparse")
    T = case.get("T", 1)
    for t in range(case["nq"] if sparse else case["B"]):
        q = s["q"][t].double().reshape(-1, c)
        if sparse:
            i = s["idx"][t]
            rows = s["kv"][0 if s["seq"] is not None else t][i[i >= 0].long()]
        else:
            rows = s["kv"][t][:int(_lens(case)[t])]
        V = _values64(rows, c, R)
        z = (q @ V.T) * scale
        if op in ("wsparse", "wdense"):
            w = torch.exp(z - s["lse"][t].double().reshape(-1, 1)).sum(0)
            if sparse:
                full = torch.zeros(case["k"], dtype=torch.float64, device=DEV)
                full[s["idx"][t] >= 0] = w
            else:
                full = s["acc"][t].double()
                full[:w.shape[0]] += w
            outs.append(full)
            continue
        zz = z if sink is None else torch.cat((z, sink[:, None]), 1)
        if zz.shape[1] == 0:
            outs.append(torch.zeros_like(q))
            extra.append(torch.full((q.shape[0],), -math.inf, dtype=torch.float64, device=DEV))
            continue
        p = torch.softmax(zz, 1)
        outs.append(p[:, :z.shape[1]] @ V)
        extra.append(torch.logsumexp(zz, 1))
    if extra:
        return torch.stack(outs), torch.stack(extra)
    return torch.stack(outs)

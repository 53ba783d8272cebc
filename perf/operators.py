"""What the 8-bit K/V cache's operators are timed and compared on: the preparation of q and k (RMS norm and
rotation), the quantising append, the read-back and the decode attention over the cache.

``run`` computes an operator in plain torch operations where ``own`` is false, and calls the package's entry points
where it is true. The cache: K8, V8 [chunks][Hkv][C][128] float8_e4m3fn with k_scale, v_scale
[chunks][Hkv][C / scale_block] float32, chunk_off the first chunk of each sequence.
"""
import math

import torch

own = False

DH = 128
MIN_EXP = -120  # the least scale is 2^-120


# ------------------------------------------------------------------------------------------------ the cases
def listed():
    return [
        # one decode token of 8 sequences: q and k of one layer, straight from a packed projection
        dict(name="prep 8 tokens", op="prep", T=8, H=16, Hkv=16, dtype="bf16", rot=128, interleaved=False, norm=True, far=1 << 20),
        # a prefill's q and k with grouped heads, half of each head rotated, positions up to 1M
        dict(name="prep 16384 tokens", op="prep", T=16384, H=32, Hkv=8, dtype="bf16", rot=64, interleaved=True, norm=True, far=1 << 20),
        # the decode step's write: one token for each of 8 sequences, 16 heads
        dict(name="append 1 token x 8", op="append", B=8, n_new=1, N=64, C=64, Hkv=16, sb=64, dtype="bf16", prep=True, ragged=False),
        # an odd, padded fp32 batch that starts and ends inside blocks
        dict(name="append 1021 tokens x 3", op="append", B=3, n_new=1021, N=96, C=16, Hkv=4, sb=16, dtype="f32", prep=False, ragged=True),
        # a prefill of 4 sequences written to the cache, K prepared in the same pass
        dict(name="append 8192 tokens x 4", op="append", B=4, n_new=8192, N=136, C=64, Hkv=16, sb=64, dtype="bf16", prep=True, ragged=False),
        # the smallest workload's kept chunks read back in fp32
        dict(name="gather 8 chunks", op="gather", B=1, N=64, C=64, k=8, Hkv=8, sb=64, dtype="f32", ragged=False),
        # the 128K workload's kept chunks read back in bf16
        dict(name="gather 256 chunks x 8", op="gather", B=8, N=2048, C=64, k=256, Hkv=16, sb=64, dtype="bf16", ragged=False),
        # ragged sequences with grouped heads, the last chunk partly filled
        dict(name="gather ragged x 5", op="gather", B=5, N=417, C=32, k=61, Hkv=4, sb=8, dtype="bf16", ragged=True),
        # the smallest workload's decode attention, fp32 queries
        dict(name="attn 8 chunks", op="attn", B=1, N=64, C=64, k=8, H=8, Hkv=8, sb=64, dtype="f32", ragged=False, dense=False),
        # the 128K workload's decode attention: 256 of 2048 chunks for 8 sequences
        dict(name="attn 256 chunks x 8", op="attn", B=8, N=2048, C=64, k=256, H=16, Hkv=16, sb=64, dtype="bf16", ragged=False, dense=False),
        # the 500K workload's kept share, with 4 query heads to a K/V head
        dict(name="attn 819 chunks x 4", op="attn", B=4, N=8192, C=64, k=819, H=32, Hkv=8, sb=64, dtype="bf16", ragged=False, dense=False),
        # a mixed batch of 32 ragged sequences, 8 query heads to a K/V head, small scale blocks
        dict(name="attn ragged x 32", op="attn", B=32, N=2048, C=64, k=276, H=32, Hkv=4, sb=16, dtype="bf16", ragged=True, dense=False),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["prep", "append", "gather", "attn", "attn"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    Hkv = rng.choice([1, 2, 4, 8, 16])
    if op == "prep":
        H = min(64, Hkv * rng.choice([1, 2, 4, 8]))
        T = _log(rng, 1, max(1, 16384 * 40 // (2 * (H + Hkv))))
        return dict(op=op, T=T, H=H, Hkv=Hkv, dtype=dtype, rot=rng.choice([128, 64, 32, 96]),
                    interleaved=rng.random() < 0.5, norm=rng.random() < 0.8, far=1 << 20)
    C = rng.choice([8, 16, 32, 64, 128, 1024])
    sb = rng.choice([s for s in (8, 16, 32, 64) if s <= C])
    B = _log(rng, 1, 40)
    rows = B * Hkv  # (sequence, head) pairs
    if op == "append":
        n_new = _log(rng, 1, max(1, 4 * 8192 * 16 // (3 * rows)))
        return dict(op=op, B=B, n_new=n_new, N=(n_new + 2 * C + 300) // C + 1, C=C, Hkv=Hkv, sb=sb, dtype=dtype,
                    prep=rng.random() < 0.5, ragged=rng.random() < 0.5)
    most = max(1, (8 * 256 * 64 * 16) // (rows * C * (1 if op == "attn" or dtype == "bf16" else 2)))
    k = _log(rng, 1, min(most, 4000))
    N = k + _log(rng, 1, max(1, 3 * k))
    N = min(N, max(k, 8 * 2048 * 64 * 16 // (rows * C)))
    if op == "gather":
        return dict(op=op, B=B, N=N, C=C, k=k, Hkv=Hkv, sb=sb, dtype=dtype, ragged=rng.random() < 0.5)
    H = min(128, Hkv * rng.choice([1, 1, 2, 4, 8, 16]))
    dense = rng.random() < 0.2
    return dict(op=op, B=B, N=k if dense else N, C=C, k=k, H=H, Hkv=Hkv, sb=sb, dtype=dtype,
                ragged=rng.random() < 0.5, dense=dense)


# ------------------------------------------------------------------------------------------------ inputs
def _dt(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _counts(case):
    """Per sequence: chunks N_b, kept chunks k_b, valid tokens. Ragged batches: between a quarter and all of N and k,
    the length ending inside the last chunk; the same shape for every seed."""
    B, N, k, C = case["B"], case["N"], case["k"], case["C"]
    if not case["ragged"]:
        return [N] * B, [k] * B, [N * C] * B
    u = torch.rand((B, 2), generator=torch.Generator().manual_seed(N * 1000003 + k)).tolist()
    n_b, k_b, len_b = [], [], []
    for x, y in u:
        f = 0.25 + 0.75 * x
        kk = max(1, int(k * f))
        nn = max(kk, int(N * f))
        n_b.append(nn)
        k_b.append(kk)
        len_b.append((nn - 1) * C + 1 + int(y * (C - 1)))
    return n_b, k_b, len_b


def _cache(chunks, Hkv, C, sb, g):
    """A filled cache: values N(0, 1) with channels and chunks of unlike size, as keys and values have them."""
    dev = "cuda"
    codes, scales = [], []
    for _ in range(2):
        c8 = torch.empty((chunks, Hkv, C, DH), dtype=torch.float8_e4m3fn, device=dev)
        sc = torch.empty((chunks, Hkv, C // sb), dtype=torch.float32, device=dev)
        channel = torch.exp(0.4 * torch.randn((Hkv, 1, DH), generator=g, device=dev))
        step = max(1, (1 << 26) // (Hkv * C * DH))
        for c0 in range(0, chunks, step):
            n = min(step, chunks - c0)
            x = torch.randn((n, Hkv, C, DH), generator=g, device=dev)
            x *= channel * torch.exp(0.5 * torch.randn((n, Hkv, 1, 1), generator=g, device=dev))
            x = x.view(n, Hkv, C // sb, sb, DH)
            s = _scale_of(x.abs().amax((3, 4)))
            sc[c0:c0 + n] = s
            c8[c0:c0 + n] = (x / s[..., None, None]).view(n, Hkv, C, DH).to(torch.float8_e4m3fn)
        codes.append(c8)
        scales.append(sc)
    return codes[0], codes[1], scales[0], scales[1]


def _inv_freq(rot):
    i = torch.arange(rot // 2, dtype=torch.float64)
    return (10000.0 ** (-2.0 * i / rot)).to(torch.float32).cuda()


def prepare(case, seed):
    op, dt, dev = case["op"], _dt(case), "cuda"
    host = torch.Generator().manual_seed(seed)
    g = torch.Generator(device=dev).manual_seed(seed)
    s = dict(case=case)
    if op == "prep":
        T, H, Hkv = case["T"], case["H"], case["Hkv"]
        # q, k and v of a token lie side by side, as a packed projection writes them
        qkv = torch.randn((T, H + 2 * Hkv, DH), generator=g, device=dev).mul_(2.0).to(dt)
        s["q"], s["k"] = qkv[:, :H], qkv[:, H:H + Hkv]
        s["pos"] = torch.randint(0, case["far"], (T,), generator=g, device=dev, dtype=torch.int32)
        s["inv_freq"] = _inv_freq(case["rot"])
        s["qw"] = 1 + 0.2 * torch.randn(DH, generator=g, device=dev) if case["norm"] else None
        s["kw"] = 1 + 0.2 * torch.randn(DH, generator=g, device=dev) if case["norm"] else None
        s["q_out"] = torch.empty((T, H, DH), dtype=dt, device=dev)
        s["k_out"] = torch.empty((T, Hkv, DH), dtype=dt, device=dev)
    elif op == "append":
        B, n, N, C, Hkv, sb = (case[x] for x in ("B", "n_new", "N", "C", "Hkv", "sb"))
        s["n_b"], s["k_b"] = [N] * B, [1] * B
        s["K8"], s["V8"], s["ks"], s["vs"] = _cache(B * N, Hkv, C, sb, g)
        qkv = torch.randn((B, n, 3 * Hkv, DH), generator=g, device=dev).mul_(1.5).to(dt)
        s["k"], s["v"] = qkv[:, :, Hkv:2 * Hkv], qkv[:, :, 2 * Hkv:]
        room = max(0, N * C - n)
        s["start"] = torch.randint(0, min(room, 300) + 1, (B,), generator=g, device=dev, dtype=torch.int32)
        s["count"] = torch.randint(0, n + 1, (B,), generator=g, device=dev, dtype=torch.int32) if case["ragged"] else None
        s["inv_freq"] = _inv_freq(DH)
        s["kw"] = 1 + 0.2 * torch.randn(DH, generator=g, device=dev)
    else:
        n_b, k_b, len_b = _counts(case)
        s["n_b"], s["k_b"] = n_b, k_b
        s["K8"], s["V8"], s["ks"], s["vs"] = _cache(sum(n_b), case["Hkv"], case["C"], case["sb"], g)
        if not case.get("dense"):
            ids = [torch.randperm(nn, generator=host)[:kk].sort().values for nn, kk in zip(n_b, k_b)]
            s["ids"] = torch.cat(ids).to(torch.int32).cuda()
        else:
            s["ids"] = None
        s["len"] = torch.tensor(len_b, dtype=torch.int32, device=dev) if case["ragged"] else None
        if op == "gather":
            rows = sum(k_b) * case["C"]
            s["K_res"] = torch.zeros((rows, case["Hkv"], DH), dtype=dt, device=dev)
            s["V_res"] = torch.zeros_like(s["K_res"])
        else:
            s["q"] = torch.randn((case["B"], case["H"], DH), generator=g, device=dev).to(dt)
            s["out"] = torch.empty((case["B"], case["H"], DH), dtype=torch.float32, device=dev)
            s["lse"] = torch.empty((case["B"], case["H"]), dtype=torch.float32, device=dev)
    if own:  # the handles that a user's program makes once: the shape, the cache's description, the workspace
        import learned_sparse_kv_decode_b200 as lsa
        if op == "prep":
            s["dims"] = lsa.Dims(1, 1, DH, case["H"], 64, N=1, k=1, kv_dtype=case["dtype"])
            s["prep"] = lsa.QkPrep(case["rot"], s["inv_freq"], s["qw"], s["kw"], 1e-6, case["interleaved"])
        else:
            off = [0]
            for nn in s["n_b"]:
                off.append(off[-1] + nn)
            s["dims"] = lsa.Dims(case["B"], 1, DH, case.get("H", case["Hkv"]), case["C"], chunk_offsets=off, k_per_seq=s["k_b"],
                                 kv_dtype=case["dtype"])
            s["cache"] = lsa.Kv8Cache(s["dims"], case["Hkv"], case["sb"], s["K8"], s["V8"], s["ks"], s["vs"])
            s["ws"] = lsa.alloc_workspace(s["dims"], kv8=s["cache"])
            s["prep"] = lsa.QkPrep(DH, s["inv_freq"], None, s["kw"], 1e-6, False) if case.get("prep") else None
    return s


# ------------------------------------------------------------------------------------------------ one pass
def run(s):
    op = s["case"]["op"]
    if own:
        import learned_sparse_kv_decode_b200 as lsa
        if op == "prep":
            lsa.lsa_qk_norm_rope(s["dims"], s["prep"], s["pos"], s["q"], s["k"], s["q_out"], s["k_out"])
            return {"q": s["q_out"], "k": s["k_out"]}
        if op == "append":
            lsa.lsa_kv8_append(s["dims"], s["cache"], s["prep"], s["k"], s["v"], s["start"], s["count"], s["ws"])
            return {"K8": s["K8"], "V8": s["V8"], "k_scale": s["ks"], "v_scale": s["vs"]}
        if op == "gather":
            lsa.lsa_kv8_gather(s["dims"], s["cache"], s["ids"], s["len"], s["K_res"], s["V_res"], s["ws"])
            return {"K": s["K_res"], "V": s["V_res"]}
        lsa.lsa_kv8_decode_attn(s["dims"], s["cache"], s["q"], s["ids"], None, s["len"], s["out"], s["lse"], s["ws"])
        return {"out": s["out"], "lse": s["lse"]}
    return {"prep": _plain_prep, "append": _plain_append, "gather": _plain_gather, "attn": _plain_attn}[op](s)


def _scale_of(amax):
    """The least power of two (2^-120 at least) that brings amax to 448 or less."""
    m, e = torch.frexp(amax)
    e = torch.where(m <= 0.875, e - 9, e - 8)
    e = torch.where(amax > 0, e, torch.full_like(e, MIN_EXP)).clamp(min=MIN_EXP)
    return torch.ldexp(torch.ones_like(amax), e)


def _norm_rope(x, pos, inv_freq, w, rot, interleaved, eps=1e-6):
    """x [..., heads, 128]; pos [...]: RMS norm with the weight w (None: no norm), then the rotation of the first rot values."""
    y = x.float()
    if w is not None:
        y = y * torch.rsqrt(y.square().mean(-1, keepdim=True) + eps) * w
    a = pos.double()[..., None] * inv_freq.double()
    c, n = torch.cos(a).float()[..., None, :], torch.sin(a).float()[..., None, :]
    if interleaved:
        y1, y2 = y[..., 0:rot:2], y[..., 1:rot:2]
        r = torch.stack((y1 * c - y2 * n, y2 * c + y1 * n), -1).flatten(-2)
    else:
        y1, y2 = y[..., :rot // 2], y[..., rot // 2:rot]
        r = torch.cat((y1 * c - y2 * n, y2 * c + y1 * n), -1)
    return torch.cat((r, y[..., rot:]), -1).to(x.dtype)


def _plain_prep(s):
    c = s["case"]
    f = lambda x, w: _norm_rope(x, s["pos"], s["inv_freq"], w, c["rot"], c["interleaved"])  # noqa: E731
    return {"q": f(s["q"], s["qw"]), "k": f(s["k"], s["kw"])}


def _plain_append(s):
    c = s["case"]
    B, n, N, C, Hkv, sb = (c[x] for x in ("B", "n_new", "N", "C", "Hkv", "sb"))
    dev = s["k"].device
    start = s["start"].long()
    i = torch.arange(n, device=dev)
    pos = start[:, None] + i
    count = s["count"].long() if s["count"] is not None else torch.full_like(start, n)
    fresh = (i < count[:, None]) & (pos < N * C)
    k = _norm_rope(s["k"], pos, s["inv_freq"], s["kw"], DH, False) if c["prep"] else s["k"]
    # the blocks that the new rows may touch, first block of each sequence first
    first = start // sb
    nblk = (n + 2 * sb - 2) // sb
    at = pos - first[:, None] * sb                                      # row within those blocks
    bi = torch.arange(B, device=dev)[:, None].expand(B, n)
    is_new = torch.zeros((B, nblk * sb), dtype=torch.bool, device=dev)
    is_new[bi[fresh], at[fresh]] = True
    row = torch.arange(nblk * sb, device=dev)
    old_rows = (row < (start - first * sb)[:, None]) & is_new.view(B, nblk, sb).any(-1)[:, :1]  # a touched first block's
    touched = is_new.view(B, nblk, sb).any(-1)
    apos = (first[:, None] * sb + row).clamp(max=N * C - 1)
    chunk, within = torch.arange(B, device=dev)[:, None] * N + apos // C, apos % C
    bchunk, bidx = chunk[:, ::sb], within[:, ::sb] // sb
    out = {}
    for name, x, codes, scales in (("K", k, s["K8"], s["ks"]), ("V", s["v"], s["V8"], s["vs"])):
        xp = torch.zeros((B, nblk * sb, Hkv, DH), device=dev)
        xp[bi[fresh], at[fresh]] = x[fresh].float()
        need = _scale_of(xp.view(B, nblk, sb, Hkv, DH).abs().amax((2, 4)))
        was = scales[bchunk, :, bidx]                                   # [B, nblk, Hkv]
        has_old = old_rows.view(B, nblk, sb).any(-1)
        now = torch.where(has_old[..., None], torch.maximum(was, need), need)
        scales[bchunk[touched], :, bidx[touched]] = now[touched]
        new = (xp.view(B, nblk, sb, Hkv, DH) / now[:, :, None, :, None]).view(B, nblk * sb, Hkv, DH)
        raw = codes.view(torch.uint8)
        raw[chunk[is_new], :, within[is_new]] = new[is_new].to(torch.float8_e4m3fn).view(torch.uint8)
        old = codes.view(torch.uint8)[chunk[old_rows], :, within[old_rows]].view(torch.float8_e4m3fn).float()
        ratio = (was / now)[:, :, None, :].expand(B, nblk, sb, Hkv).reshape(B, nblk * sb, Hkv)[old_rows]
        raw[chunk[old_rows], :, within[old_rows]] = (old * ratio[..., None]).to(torch.float8_e4m3fn).view(torch.uint8)
        out[name + "8"], out[name.lower() + "_scale"] = codes, scales
    return out


def _chunk_index(s):
    """Global chunk of each kept chunk [sum k_b], its local id, and its sequence."""
    dev = s["K8"].device
    counts = s["n_b"] if s["ids"] is None else s["k_b"]
    counts_t = torch.tensor(counts, device=dev)
    n_t = torch.tensor(s["n_b"], device=dev)
    seq = torch.repeat_interleave(torch.arange(len(counts), device=dev), counts_t, output_size=sum(counts))
    place = torch.arange(sum(counts), device=dev) - (counts_t.cumsum(0) - counts_t)[seq]
    ids = s["ids"].long() if s["ids"] is not None else place
    return (n_t.cumsum(0) - n_t)[seq] + ids, ids, seq, place, max(counts)


def _deq(codes, scales, chunk):
    """[kept][Hkv][C][128] float32 values of the given chunks."""
    x = codes.view(torch.uint8)[chunk].view(torch.float8_e4m3fn).float()
    n, h, c, d = x.shape
    sc = scales[chunk]
    return (x.view(n, h, sc.shape[2], -1, d) * sc[..., None, None]).view(n, h, c, d)


def _valid(s, ids, seq):
    """[kept][C]: whether a token lies before its sequence's length."""
    C = s["case"]["C"]
    t = ids[:, None] * C + torch.arange(C, device=ids.device)
    return torch.ones_like(t, dtype=torch.bool) if s["len"] is None else t < s["len"].long()[seq][:, None]


def _plain_gather(s):
    chunk, ids, seq, _, _ = _chunk_index(s)
    ok = _valid(s, ids, seq).view(-1, 1, 1)
    out = {}
    for name, codes, scales, res in (("K", s["K8"], s["ks"], s["K_res"]), ("V", s["V8"], s["vs"], s["V_res"])):
        x = _deq(codes, scales, chunk).permute(0, 2, 1, 3).reshape(res.shape).to(res.dtype)
        out[name] = torch.where(ok, x, res)
    return out


def _plain_attn(s):
    c = s["case"]
    B, H, Hkv, C = c["B"], c["H"], c["Hkv"], c["C"]
    chunk, ids, seq, place, most = _chunk_index(s)
    ok = torch.zeros((B, most, C), dtype=torch.bool, device=chunk.device)
    ok[seq, place] = _valid(s, ids, seq)
    q = s["q"].float().view(B, Hkv, H // Hkv, DH)
    k = _deq(s["K8"], s["ks"], chunk)                                   # [kept][Hkv][C][128]
    logit = torch.full((B, most, Hkv, H // Hkv, C), -math.inf, device=chunk.device)
    logit[seq, place] = torch.matmul(q[seq], k.transpose(-1, -2)) / math.sqrt(DH)
    del k
    logit = logit.masked_fill(~ok[:, :, None, None, :], -math.inf)
    m = logit.amax((1, 4), keepdim=True)
    p = torch.exp(logit - m.masked_fill(m == -math.inf, 0.0))
    total = p.sum((1, 4))
    v = _deq(s["V8"], s["vs"], chunk)
    part = torch.matmul(p[seq, place], v)                               # [kept][Hkv][group][128]
    o = torch.zeros((B, most, Hkv, H // Hkv, DH), device=chunk.device)
    o[seq, place] = part
    o = o.sum(1) / total[..., None].clamp(min=1e-38)
    lse = torch.log(total) + m.view(total.shape)
    return {"out": o.view(B, H, DH), "lse": lse.view(B, H)}


# ------------------------------------------------------------------------------------------------ work
def work(case):
    op, es = case["op"], 2 if case["dtype"] == "bf16" else 4
    if op == "prep":
        rows = case["T"] * (case["H"] + case["Hkv"])
        return {"bytes": rows * DH * es * 2 + 4 * case["T"], "flops": rows * DH * 8}
    if op == "append":
        rows = case["B"] * case["n_new"] * case["Hkv"] * 2 * (0.5 if case["ragged"] else 1.0)
        return {"bytes": rows * DH * (es + 1) + rows / case["sb"] * 4, "flops": rows * DH * (10 if case["prep"] else 2)}
    kept = (case["N"] if case.get("dense") else case["k"]) * case["B"] * (0.62 if case["ragged"] else 1.0)
    rows = kept * case["C"] * case["Hkv"] * 2
    if op == "gather":
        return {"bytes": rows * DH * (1 + es) + rows / case["sb"] * 4 + kept * 4, "flops": rows * DH}
    q = case["B"] * case["H"] * DH
    return {"bytes": rows * DH + rows / case["sb"] * 4 + kept * 4 + q * (es + 4), "flops": 4 * DH * kept * case["C"] * case["H"]}


# ------------------------------------------------------------------------------------------------ in 64 bits
def _round_e4m3(y):
    """Values of y (double, |y| <= 448) rounded to the nearest e4m3 value, ties to even."""
    e = torch.frexp(y)[1].double() - 1
    step = torch.exp2(e.clamp(min=-6) - 3)
    return torch.round(y / step) * step


def _exact_rope(x, pos, inv_freq, w, rot, interleaved):
    y = x.double()
    if w is not None:
        y = y / torch.sqrt((y * y).sum(-1, keepdim=True) / DH + 1e-6) * w.double()
    z = y.clone()
    for i in range(rot // 2):
        a = pos.double() * float(inv_freq[i])
        co, si = torch.cos(a)[..., None], torch.sin(a)[..., None]
        p, r = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
        z[..., p] = y[..., p] * co - y[..., r] * si
        z[..., r] = y[..., r] * co + y[..., p] * si
    return z


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "prep":
        f = lambda x, w: _exact_rope(x, s["pos"], s["inv_freq"], w, case["rot"], case["interleaved"])  # noqa: E731
        return {"q": f(s["q"], s["qw"]), "k": f(s["k"], s["kw"])}
    if op == "append":
        return _exact_append(s)
    sb, C = case["sb"], case["C"]
    off, kept = 0, 0
    outs, sums, res = [], [], {"K": [], "V": []}
    for b, (nn, kk) in enumerate(zip(s["n_b"], s["k_b"])):
        ids = torch.arange(nn, device="cuda") if s["ids"] is None else s["ids"][kept:kept + kk].long()
        t = (ids[:, None] * C + torch.arange(C, device="cuda")).view(-1)
        ok = t < (nn * C if s["len"] is None else int(s["len"][b]))
        heads = []
        for h in range(case["Hkv"]):
            kv = []
            for codes, scales in ((s["K8"], s["ks"]), (s["V8"], s["vs"])):
                x = codes[off:off + nn, h].view(torch.uint8)[ids].view(torch.float8_e4m3fn).double()
                kv.append((x * scales[off:off + nn, h][ids].double().repeat_interleave(sb, 1)[..., None]).view(-1, DH))
            if op == "gather":
                heads.append([torch.where(ok[:, None], x, 0.0) for x in kv])
                continue
            g = case["H"] // case["Hkv"]
            q = s["q"][b, h * g:(h + 1) * g].double()
            logit = (q @ kv[0][ok].T) / math.sqrt(DH)
            sums.append(torch.logsumexp(logit, -1))
            outs.append(torch.softmax(logit, -1) @ kv[1][ok])
        if op == "gather":
            for name, j in (("K", 0), ("V", 1)):
                res[name].append(torch.stack([x[j] for x in heads], 1).to(torch.float32))
        off, kept = off + nn, kept + kk
    if op == "gather":  # a code times a power of two: the float32 is the value itself
        return {n: torch.cat(v) for n, v in res.items()}
    return {"out": torch.cat(outs).view(case["B"], case["H"], DH), "lse": torch.cat(sums).view(case["B"], case["H"])}


def _exact_append(s):
    case = s["case"]
    N, C, sb, n = case["N"], case["C"], case["sb"], case["n_new"]
    if case["B"] * (n // sb + 2) > 8000:  # some ten seconds of small steps
        return None
    out = {}
    for name, x, codes, scales in (("K", s["k"], s["K8"], s["ks"]), ("V", s["v"], s["V8"], s["vs"])):
        c64, s64 = codes.float(), scales.clone().double()
        for b in range(case["B"]):
            start = int(s["start"][b])
            count = n if s["count"] is None else int(s["count"][b])
            rows = x[b, :count].double()
            if name == "K" and case["prep"]:
                pos = torch.arange(start, start + count, device="cuda")
                rows = _exact_rope(x[b, :count], pos, s["inv_freq"], s["kw"], DH, False).to(x.dtype).double()
            end = min(start + count, N * C)
            for blk in range(start // sb, (end + sb - 1) // sb if end > start else 0):
                lo, hi = max(blk * sb, start), min(blk * sb + sb, end)
                r = rows[lo - start:hi - start].transpose(0, 1)         # [Hkv][rows][128]
                top = r.abs().amax((1, 2))
                e = torch.ceil(torch.log2(torch.clamp(top / 448, min=2.0 ** -130)))
                sc = torch.exp2(e.clamp(min=MIN_EXP))
                sc = torch.where(top > 448 * sc, 2 * sc, torch.where(top <= 224 * sc, sc / 2, sc)).clamp(min=2.0 ** MIN_EXP)
                chunk, w0 = b * N + blk * sb // C, blk * sb % C
                if lo > blk * sb:
                    was = s64[chunk, :, w0 // sb].clone()
                    sc = torch.maximum(sc, was)
                    j = slice(w0, w0 + lo - blk * sb)
                    c64[chunk, :, j] = _round_e4m3(c64[chunk, :, j].double() * (was / sc)[:, None, None]).float()
                s64[chunk, :, w0 // sb] = sc
                c64[chunk, :, w0 + lo - blk * sb:w0 + hi - blk * sb] = _round_e4m3(r / sc[:, None, None]).float()
        out[name + "8"], out[name.lower() + "_scale"] = c64, s64
    return out

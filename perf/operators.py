"""Timed cases of the 8-bit latent cache and of chunks of new tokens over paged caches.

Four operators, at the full shapes (64 x 128 indexer, 128 query heads, latent rows of 512 values
and 64 rotary dims, pages of 64 tokens):

  append   the new tokens' indexer keys (e4m3, one fp32 scale a token) and latent rows (e4m3 with
           one power-of-two scale per 128 values, rotary dims kept in bf16) written into the
           paged caches, one token per sequence or a chunk of several
  read     ranges of the 8-bit cache read back as packed bf16 rows
  attn     attention of every new token over its selected keys (output and log-sum-exp), over the
           8-bit cache or the bf16 one, for single tokens and for chunks
  scores   the indexer's scores of a chunk's rows against every prior key of the paged key cache

A case's ``new`` and ``ctx`` list, per sequence, the new tokens and the context length that
already counts them.  ``run`` computes the plain form in torch, or with ``own`` makes the calls
of this repository's package.
"""
import math

import numpy as np
import torch

own = False

H_I, D_I = 64, 128
H, D_QK, D_V = 128, 576, 512
ROPE = D_QK - D_V
GROUP = 128
GROUPS = D_V // GROUP
ROW = D_V + 4 * GROUPS + 2 * ROPE        # bytes of one 8-bit cache row: codes, scales, rotary dims
PAGE = 64
SIGMA = 1.0 / math.sqrt(D_QK)
E_MIN, E_MAX = -100, 119                 # exponents of a group's power-of-two scale


def _ints(text):
    return [int(x) for x in text.split(",")]


# ------------------------------------------------------------------------------------ cases

def listed():
    return [
        # one sequence's next token: pure latency
        dict(name="append_1", op="append", new="1", ctx="4096"),
        # one decode step of a batch (the batch of the paged 128k decode workload)
        dict(name="append_b64", op="append", new=",".join(["1"] * 64),
             ctx=",".join(str(2048 + 97 * i) for i in range(64))),
        # chunks of several prompts entering the caches in one call, odd lengths and one token
        dict(name="append_chunks", op="append", new="4096,777,1,63,8192,2050,333",
             ctx="16384,777,9000,64,8192,5001,20000"),
        # a short prefix and its odd tail read back (a cached prompt handed to a dense pass)
        dict(name="read_short", op="read", ctx="1000,65,1"),
        # whole contexts moved out of the cache (two of 64k, ragged others)
        dict(name="read_long", op="read", ctx="65536,65536,32768,9999,50001"),
        # one sequence's next token over 32k: few rows, the work split over the selection
        dict(name="attn_token_b1", op="attn", cache="q8", topk=2048, new="1", ctx="32768"),
        # a decode step of 64 sequences of 32k
        dict(name="attn_token_b64", op="attn", cache="q8", topk=2048, new=",".join(["1"] * 64),
             ctx=",".join(["32768"] * 64)),
        # mixed step: single tokens, drafted tokens being verified and prompt chunks, contexts
        # below and above the selection
        dict(name="attn_mixed", op="attn", cache="q8", topk=2048, new="1,4,130,37,64,1,257,8",
             ctx="5000,8191,130,20011,2100,1,1500,40000"),
        # one large prompt chunk over a long context, 8-bit and bf16 caches
        dict(name="attn_chunk_q8", op="attn", cache="q8", topk=2048, new="2048", ctx="32768"),
        dict(name="attn_chunk_bf16", op="attn", cache="bf16", topk=2048, new="1000",
             ctx="32768"),
        # a prompt chunk's indexer scores over 64k
        dict(name="scores_chunk", op="scores", new="512", ctx="65536"),
        # drafted tokens of 32 sequences scored before their verification
        dict(name="scores_drafts", op="scores", new=",".join(["4"] * 32),
             ctx=",".join(str(4099 + 128 * i) for i in range(32))),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "read", "attn", "attn", "scores"])
    batch = _log_int(rng, 1, 32)
    if op == "append":
        new = [_log_int(rng, 1, max(1, 12000 // batch)) for _ in range(batch)]
        if rng.random() < 0.3:
            new = [1] * batch
        ctx = [n + (0 if rng.random() < 0.3 else _log_int(rng, 1, 8000)) for n in new]
        return dict(op=op, new=",".join(map(str, new)), ctx=",".join(map(str, ctx)))
    if op == "read":
        ctx = [_log_int(rng, 1, max(1, 220000 // batch)) for _ in range(batch)]
        return dict(op=op, ctx=",".join(map(str, ctx)))
    if op == "attn":
        new = [_log_int(rng, 1, max(1, 1800 // batch)) for _ in range(batch)]
        if rng.random() < 0.3:
            new = [1] * batch
        ctx = [n + (0 if rng.random() < 0.2 else _log_int(rng, 1, 30000)) for n in new]
        return dict(op=op, cache=rng.choice(["q8", "q8", "bf16"]),
                    topk=64 * rng.choice([1, 5, 16, 31, 32, 32, 32]),
                    new=",".join(map(str, new)), ctx=",".join(map(str, ctx)))
    # the products of all sequences' longest rows and contexts stay below the largest listed
    longest = _log_int(rng, 1, max(1, 400 // batch))
    new = [max(1, longest - rng.randrange(0, max(1, longest // 2))) for _ in range(batch)]
    top = max(256, min(60000, 24000000 // (longest * batch), 600000 // batch))
    ctx = [n + _log_int(rng, 1, top - 1) for n in new]
    return dict(op=op, new=",".join(map(str, new)), ctx=",".join(map(str, ctx)))


def _geometry(case):
    ctx = _ints(case["ctx"])
    new = _ints(case["new"]) if "new" in case else list(ctx)
    return new, ctx


def _keys_seen(new, ctx):
    """Keys seen by every new token, summed, and the per-row list."""
    return [c - n + i + 1 for n, c in zip(new, ctx) for i in range(n)]


def work(case):
    new, ctx = _geometry(case)
    rows = sum(new)
    if case["op"] == "append":
        return {"bytes": rows * (4 * D_I + 2 * D_QK + D_I + 4 + ROW), "flops": 0}
    if case["op"] == "read":
        return {"bytes": rows * (ROW + 2 * D_QK), "flops": 0}
    seen = _keys_seen(new, ctx)
    if case["op"] == "scores":
        return {"bytes": sum(ctx) * (D_I + 4) + rows * H_I * (D_I + 8) + 4 * sum(seen),
                "flops": 2 * H_I * D_I * sum(seen)}
    sel = [min(s, case["topk"]) for s in seen]
    row_bytes = ROW if case["cache"] == "q8" else 2 * D_QK
    # distinct rows read: the expected union of a sequence's random selections
    uniq = 0.0
    at = 0
    for n, c in zip(new, ctx):
        left = 1.0
        for i in range(n):
            left *= 1.0 - sel[at + i] / max(seen[at + i], 1)
        uniq += c * (1.0 - left)
        at += n
    return {"bytes": int(uniq * row_bytes) + rows * (H * (2 * D_QK + 2 * D_V + 4) + 4 * case["topk"]),
            "flops": 2 * H * (D_QK + D_V) * sum(sel)}


# ------------------------------------------------------------------------------ input making

def _group_scale(x):
    """The smallest power of two s with max|x| <= 448 s, over the last axis (1 for all zeros)."""
    amax = x.abs().amax(dim=-1)
    m, e = torch.frexp(amax)                       # amax = m 2^e, m in [0.5, 1); 448 = 0.875 2^9
    e = (e - torch.where(m <= 0.875, 9, 8)).clamp(E_MIN, E_MAX)
    s = torch.ldexp(torch.ones_like(amax), e)
    return torch.where(amax > 0, s, torch.ones_like(s))


def _pack_rows(latent):
    """bf16 latent rows [n, D_QK] -> 8-bit cache rows, uint8 [n, ROW]."""
    x = latent[:, :D_V].float().reshape(-1, GROUPS, GROUP)
    s = _group_scale(x)
    codes = (x / s.unsqueeze(-1)).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
    return torch.cat([codes.reshape(-1, D_V).view(torch.uint8), s.view(torch.uint8),
                      latent[:, D_V:].contiguous().view(torch.uint8)], dim=1)


def _key_scale(x):
    amax = x.abs().amax(dim=-1)
    return torch.where(amax > 0, amax / 448.0, torch.ones_like(amax))


def _latents(n, g):
    """Latent rows: Gaussian values whose size differs from token to token."""
    size = torch.exp(0.3 * torch.randn(n, 1, generator=g, device="cuda"))
    return (torch.randn(n, D_QK, generator=g, device="cuda") * size).to(torch.bfloat16)


def _indexer_inputs(rows, g):
    """e4m3 indexer queries [rows, H_I, D_I] with their scales and head weights."""
    x = torch.randn(rows, H_I, D_I, generator=g, device="cuda")
    s = _key_scale(x.reshape(rows, -1))
    q8 = (x / s[:, None, None]).clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8)
    return (q8.contiguous(), s.unsqueeze(1).expand(-1, H_I).contiguous(),
            torch.rand(rows, H_I, generator=g, device="cuda"))


def prepare(case, seed):
    new, ctx = _geometry(case)
    g = torch.Generator(device="cuda").manual_seed(seed)
    batch, rows = len(ctx), sum(new)
    i32 = dict(dtype=torch.int32, device="cuda")
    # pages of every sequence scattered over a pool with a few spare pages
    pages = [(c + PAGE - 1) // PAGE for c in ctx]
    total = sum(pages) + 3
    perm = torch.randperm(total, generator=g, device="cuda").to(torch.int32)
    table = torch.zeros(batch, max(pages), **i32)
    at = 0
    for b, n in enumerate(pages):
        table[b, :n] = perm[at:at + n]
        at += n
    pool = total * PAGE
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    st = dict(op=case["op"], rows=rows, pool=pool, cu=torch.tensor(cu, **i32),
              ctx=torch.tensor(ctx, **i32), table=table, longest=max(ctx), lens=ctx)
    if case["op"] == "append":
        st["k_new"] = 3.0 * torch.randn(rows, D_I, generator=g, device="cuda")
        st["kv_new"] = _latents(rows, g)
        st["k8"] = torch.zeros(pool, D_I, dtype=torch.uint8, device="cuda")
        st["k_scale"] = torch.zeros(pool, device="cuda")
        st["kv8"] = torch.zeros(pool, ROW, dtype=torch.uint8, device="cuda")
    if case["op"] == "read" or case.get("cache") == "q8":
        kv8 = torch.empty(pool, ROW, dtype=torch.uint8, device="cuda")
        for r in range(0, pool, 1 << 18):
            n = min(1 << 18, pool - r)
            kv8[r:r + n] = _pack_rows(_latents(n, g))
        st["kv8"] = kv8
    if case["op"] == "attn":
        if case["cache"] == "bf16":
            st["kv"] = torch.cat([_latents(min(1 << 18, pool - r), g)
                                  for r in range(0, pool, 1 << 18)])
        st["q"] = torch.randn(rows, H, D_QK, generator=g, device="cuda").to(torch.bfloat16)
        # a selection as a top-k leaves it: distinct keys in increasing order, then -1
        topk = case["topk"]
        seen = torch.tensor(_keys_seen(new, ctx), device="cuda")
        width = max(max(ctx), topk)
        idx = torch.empty(rows, topk, **i32)
        for r in range(0, rows, 512):
            lim = seen[r:r + 512, None]
            key = torch.rand(lim.shape[0], width, generator=g, device="cuda")
            key = torch.where(torch.arange(width, device="cuda") < lim, key, 2.0)
            pick = key.topk(topk, dim=1, largest=False).indices
            pick = torch.where(pick < lim, pick, width).sort(dim=1).values
            idx[r:r + 512] = torch.where(pick < width, pick, -1).to(torch.int32)
        st["idx"], st["topk"] = idx, topk
        if own:
            st["out"] = torch.empty(rows, H, D_V, dtype=torch.bfloat16, device="cuda")
            st["lse"] = torch.empty(rows, H, device="cuda")
    if case["op"] == "scores":
        st["q8"], st["q_scale"], st["w"] = _indexer_inputs(rows, g)
        k = torch.randn(pool, D_I, generator=g, device="cuda")
        s = _key_scale(k)
        st["k8"] = (k / s[:, None]).clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8)
        st["k_scale"] = s
        st["ld"] = (max(ctx) + 3) // 4 * 4
        st["slab"] = torch.zeros(rows, st["ld"], device="cuda")
        # the padded view of the rows that the plain form works on
        st["most"] = max(new)
    if own:
        import sparse_attention_long_04_b200 as dsa
        single = all(n == 1 for n in new) and case["op"] != "read"
        dims = dict(h_idx=H_I, d_idx=D_I, h=H, d_qk=D_QK, d_v=D_V, topk=case.get("topk", 2048),
                    softmax_scale=SIGMA, num_kv_rows=pool, block_table=table,
                    seq_lens=st["ctx"], max_seqlen=max(ctx))
        if single or case["op"] == "read":
            st["pb"] = dsa.make_problem(mode="decode", seqlens=ctx, **dims)
        else:
            st["pb"] = dsa.make_problem(mode="chunk", seqlens=new, cu_seqlens=st["cu"], **dims)
        st["status"] = torch.zeros(1, **i32)
        if case["op"] == "read":
            st["packed"] = torch.empty(rows, D_QK, dtype=torch.bfloat16, device="cuda")
        if case["op"] == "attn":
            size = (dsa.dsa_sparse_mla_q8_workspace_size if case["cache"] == "q8"
                    else dsa.dsa_sparse_mla_workspace_size)
            st["ws_bytes"] = size(st["pb"], rows)
            st["ws"] = torch.empty(max(16, st["ws_bytes"]), dtype=torch.uint8, device="cuda")
    return st


# ------------------------------------------------------------------------------- the operators

def _rows_of(st):
    """Sequence and position of every new token (or, for a read, of every key read)."""
    r = torch.arange(st["rows"], device="cuda")
    seq = torch.searchsorted(st["cu"][1:].contiguous(), r.to(torch.int32), right=True)
    first = st["ctx"] - (st["cu"][1:] - st["cu"][:-1])
    return seq, r - st["cu"][seq] + first[seq]


def _physical(st, seq, pos):
    return st["table"][seq, pos // PAGE].long() * PAGE + pos % PAGE


def _cache_views(st):
    kv8 = st["kv8"]
    return [st["k8"].view(torch.float8_e4m3fn), st["k_scale"],
            kv8[:, :D_V].view(torch.float8_e4m3fn), kv8[:, D_V:D_V + 4 * GROUPS].view(torch.float32),
            kv8[:, D_V + 4 * GROUPS:].view(torch.bfloat16)]


def _unpack(rows):
    """8-bit cache rows [..., ROW] -> fp32 values [..., D_QK]."""
    codes = rows[..., :D_V].contiguous().view(torch.float8_e4m3fn).float()
    scale = rows[..., D_V:D_V + 4 * GROUPS].contiguous().view(torch.float32)
    rope = rows[..., D_V + 4 * GROUPS:].contiguous().view(torch.bfloat16).float()
    return torch.cat([codes * scale.repeat_interleave(GROUP, dim=-1), rope], dim=-1)


def _plain_append(st):
    phys = _physical(st, *_rows_of(st))
    s = _key_scale(st["k_new"])
    st["k8"][phys] = (st["k_new"] / s[:, None]).clamp(-448.0, 448.0).to(
        torch.float8_e4m3fn).view(torch.uint8)
    st["k_scale"][phys] = s
    st["kv8"][phys] = _pack_rows(st["kv_new"])
    return _cache_views(st)


def _plain_read(st):
    return _unpack(st["kv8"][_physical(st, *_rows_of(st))]).to(torch.bfloat16)


def _plain_attn(st):
    seq, _ = _rows_of(st)
    idx = st["idx"].long()
    phys = _physical(st, seq[:, None], idx.clamp_min(0))
    kv = _unpack(st["kv8"][phys]) if "kv8" in st else st["kv"][phys].float()
    logit = torch.matmul(st["q"].float(), kv.transpose(1, 2)) * SIGMA
    logit = logit.masked_fill((idx < 0).unsqueeze(1), -math.inf)
    m = logit.amax(dim=-1, keepdim=True)
    p = torch.exp(logit - torch.where(m == -math.inf, 0.0, m))
    l = p.sum(dim=-1, keepdim=True)
    out = torch.matmul(p, kv[..., :D_V]) / torch.where(l > 0, l, 1.0)
    return out.to(torch.bfloat16), (m + torch.log(l)).squeeze(-1)


def _plain_scores(st):
    # rows padded per sequence: [batch, most, ...] against the sequence's keys [batch, keys, D_I]
    batch, most, ld = st["ctx"].shape[0], st["most"], st["ld"]
    seq, pos = _rows_of(st)
    slot = seq * most + torch.arange(st["rows"], device="cuda") - st["cu"][seq]
    q = torch.zeros(batch * most, H_I, D_I, device="cuda")
    q[slot] = st["q8"].view(torch.float8_e4m3fn).float()
    s = torch.arange(ld, device="cuda")
    page = st["table"][:, (s // PAGE).clamp_max(st["table"].shape[1] - 1)].long()
    phys = page * PAGE + s % PAGE
    k = st["k8"].view(torch.float8_e4m3fn)[phys].float()                # [batch, ld, D_I]
    dots = torch.matmul(q.reshape(batch, most * H_I, D_I), k.transpose(1, 2)).relu_()
    c = torch.zeros(batch * most, H_I, device="cuda")
    c[slot] = st["w"] * st["q_scale"]
    score = torch.matmul(c.reshape(batch * most, 1, H_I),
                         dots.reshape(batch * most, H_I, ld)).squeeze(1)
    score = score[slot] * st["k_scale"][phys][seq]
    return torch.where(s <= pos[:, None], score, st["slab"])


def run(st):
    if not own:
        return {"append": _plain_append, "read": _plain_read, "attn": _plain_attn,
                "scores": _plain_scores}[st["op"]](st)
    import sparse_attention_long_04_b200 as dsa
    if st["op"] == "append":
        dsa.check(dsa.dsa_cache_append_q8(st["pb"], st["k_new"], st["kv_new"], st["k8"],
                                          st["k_scale"], st["kv8"], st["status"]))
        return _cache_views(st)
    if st["op"] == "read":
        dsa.check(dsa.dsa_cache_read_q8(st["pb"], st["kv8"], None, st["cu"], st["rows"],
                                        st["packed"], st["status"]))
        return st["packed"]
    if st["op"] == "attn":
        call, cache = ((dsa.dsa_sparse_mla_fwd_q8, st["kv8"]) if "kv8" in st
                       else (dsa.dsa_sparse_mla_fwd, st["kv"]))
        dsa.check(call(st["pb"], st["q"], cache, st["idx"], 0, st["rows"], st["out"], st["lse"],
                       st["ws"], st["ws_bytes"], st["status"]))
        return st["out"], st["lse"]
    dsa.check(dsa.dsa_indexer_scores(st["pb"], st["q8"], st["q_scale"], st["w"], st["k8"],
                                     st["k_scale"], 0, st["rows"], st["slab"], st["ld"],
                                     st["status"]))
    return st["slab"]


# ------------------------------------------------------------------------- 64-bit definitions

def _e4m3_values(y):
    """The e4m3 value nearest to each y (ties to even, saturating), in float64."""
    y = np.clip(y, -448.0, 448.0)
    mag = np.maximum(np.abs(y), 2.0 ** -6)
    step = 2.0 ** (np.floor(np.log2(mag)) - 3)
    return np.rint(y / step) * step


def _decode_bytes(codes):
    """Values of e4m3 bytes, in float64."""
    b = np.arange(256)
    e, m = (b >> 3) & 15, b & 7
    v = np.where(e == 0, m * 2.0 ** -9, (1.0 + m / 8.0) * 2.0 ** (e - 7.0))
    return np.where(b >= 128, -v, v)[codes]


def _host_geometry(st):
    """Physical rows of every sequence's logical positions, on the host."""
    table = st["table"].cpu().numpy().astype(np.int64)
    return [table[b, np.arange(n) // PAGE] * PAGE + np.arange(n) % PAGE
            for b, n in enumerate(st["lens"])]


def exact(case, seed):
    new, ctx = _geometry(case)
    st = prepare(case, seed)
    where = _host_geometry(st)
    if case["op"] == "append":
        phys = np.concatenate([w[c - n:c] for w, n, c in zip(where, new, ctx)])
        pool = st["pool"]
        k = st["k_new"].double().cpu().numpy()
        top = np.abs(k).max(axis=1)
        s = np.where(top > 0, top / 448.0, 1.0).astype(np.float32).astype(np.float64)
        k8, ks = np.zeros((pool, D_I)), np.zeros(pool)
        k8[phys], ks[phys] = _e4m3_values(k / s[:, None]), s
        x = st["kv_new"].double().cpu().numpy()
        lat = x[:, :D_V].reshape(-1, GROUPS, GROUP)
        top = np.abs(lat).max(axis=2)
        e = np.clip(np.ceil(np.log2(np.where(top > 0, top, 448.0) / 448.0)), E_MIN, E_MAX)
        gs = 2.0 ** e
        codes, scales, rope = np.zeros((pool, D_V)), np.zeros((pool, GROUPS)), np.zeros((pool, ROPE))
        codes[phys] = _e4m3_values(lat / gs[:, :, None]).reshape(-1, D_V)
        scales[phys], rope[phys] = gs, x[:, D_V:]
        return [k8, ks, codes, scales, rope]

    def latent(rows):                                   # float64 values of 8-bit cache rows
        raw = st["kv8"][torch.as_tensor(rows, device="cuda")].cpu().numpy()
        v = _decode_bytes(raw[:, :D_V])
        s = np.ascontiguousarray(raw[:, D_V:D_V + 4 * GROUPS]).view(np.float32).astype(np.float64)
        bits = np.ascontiguousarray(raw[:, D_V + 4 * GROUPS:]).view(np.uint16).astype(np.uint32)
        rope = (bits << 16).view(np.float32).astype(np.float64)
        return np.concatenate([v * np.repeat(s, GROUP, axis=1), rope], axis=1)

    if case["op"] == "read":
        return np.concatenate([latent(w) for w in where])
    if case["op"] == "attn":
        out = torch.zeros(st["rows"], H, D_V, dtype=torch.float64, device="cuda")
        lse = torch.full((st["rows"], H), -math.inf, dtype=torch.float64, device="cuda")
        r = 0
        for b, n in enumerate(new):
            if "kv8" in st:
                keys = torch.as_tensor(latent(where[b]), device="cuda")
            else:
                keys = st["kv"][torch.as_tensor(where[b], device="cuda")].double()
            for i in range(n):
                sel = st["idx"][r]
                sel = sel[sel >= 0].long()
                if sel.numel():
                    kv = keys[sel]
                    logit = st["q"][r].double() @ kv.T / math.sqrt(D_QK)
                    lse[r] = torch.logsumexp(logit, dim=1)
                    out[r] = torch.exp(logit - lse[r][:, None]) @ kv[:, :D_V]
                r += 1
        return out, lse
    slab = torch.zeros(st["rows"], st["ld"], dtype=torch.float64, device="cuda")
    q = torch.as_tensor(_decode_bytes(st["q8"].cpu().numpy()), device="cuda")
    c = st["w"].double() * st["q_scale"].double()
    r = 0
    for b, n in enumerate(new):
        rows = torch.as_tensor(where[b], device="cuda")
        k = torch.as_tensor(_decode_bytes(st["k8"][rows].cpu().numpy()), device="cuda")
        ks = st["k_scale"][rows].double()
        for i in range(n):
            seen = ctx[b] - n + i + 1
            dots = torch.relu(q[r] @ k[:seen].T)
            slab[r, :seen] = (c[r] @ dots) * ks[:seen]
            r += 1
    return slab

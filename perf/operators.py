"""Cases and plain forms of the 4-bit latent cache and of the batch plan.

The operators (declared in include/dsa.h):

  plan    dsa_batch_plan: block table, slot map and row map of one step, from the
          requests' lengths, with the pages taken from and given back to a free list
  append  dsa_cache_append_slots into a cache with 4-bit latents, then
          dsa_cache_read of the same slots (what a later step sees of the tokens)
  read    dsa_cache_read: gather and dequantise cached tokens (the un-absorbed
          prefill over a cached context, a cache migration)
  attn    dsa_sparse_mla_fwd over a cache with 4-bit latents

``own`` False computes them in elementary torch operations, True calls the library.

A packed latent row (DSA_INT4) of d_c latent and d_r RoPE dims holds
  bytes [0, d_c/2)          codes: 4-bit two's complement; in each little-endian
                            32-bit word the low half holds the four even dims of
                            eight (nibble i: dim 2i), the high half the odd ones
  bytes [d_c/2, +2 d_r)     the RoPE key in bf16
  then d_c/16 bytes         one scale per 16 latent dims: an unsigned 8-bit float
                            with 5 exponent and 3 mantissa bits, the fp16 number
                            whose bit pattern is the byte shifted left by 7
"""
import math

import numpy as np
import torch

own = False

D_C, D_R, D_IDX = 512, 64, 128
ROW = D_C // 2 + 2 * D_R + D_C // 16
SM_SCALE = 1.0 / math.sqrt(D_C + D_R)
GROUP = 16
SCALE_MAX_CODE = 0xF7
DEV = "cuda"


# ---------------------------------------------------------------------------- cases

def listed():
    return [
        # one decoding step of a busy server: 256 requests with a token each
        dict(name="plan decode 256", op="plan", seqs=256, lo=1, hi=1, ctx=131072, page=64, pad=0, free=512, release=0.0),
        # decoding requests beside chunks of prompts, with finished requests handing their pages back
        dict(name="plan mixed 509", op="plan", seqs=509, lo=0, hi=67, ctx=32768, page=64, pad=1003, free=900, release=0.1),
        # the largest: thousands of requests and a chunked prefill of 128K tokens in one plan
        dict(name="plan prefill 4096", op="plan", seqs=4096, lo=1, hi=61, ctx=16384, page=64, pad=4096, free=6000, release=0.02),
        # the new tokens of one decoding step (16 sequences of two tokens)
        dict(name="append decode 32", op="append", n=32, tokens=262144, page=64),
        # a whole 64K prompt
        dict(name="append prefill 65536", op="append", n=65536, tokens=131072, page=64),
        # a short shared prefix, a ragged number of tokens with a few that are not cached
        dict(name="read 5003", op="read", n=5003, tokens=262144, page=64, holes=7),
        # a 128K context read back for an un-absorbed prefill chunk
        dict(name="read 131072", op="read", n=131072, tokens=262144, page=64, holes=0),
        # one request, a short context: latency
        dict(name="attn single 517", op="attn", seqs=1, rows=1, ctx_lo=517, ctx_hi=517, heads=128, topk=2048, page=64, pad=0),
        # decoding, 32 sequences of 8K to 16K tokens, contiguous
        dict(name="attn decode 16K", op="attn", seqs=32, rows=1, ctx_lo=8192, ctx_hi=16384, heads=128, topk=2048, page=0, pad=0),
        # decoding with two tokens a sequence, 96K to 128K, paged
        dict(name="attn decode 128K paged", op="attn", seqs=16, rows=2, ctx_lo=98304, ctx_hi=131072, heads=128, topk=2048, page=64, pad=0),
        # one rank of eight that share the heads, short and odd contexts, a padded batch
        dict(name="attn heads 16", op="attn", seqs=61, rows=1, ctx_lo=3, ctx_hi=4099, heads=16, topk=1000, page=64, pad=3),
        # a 2048-token chunk of an 8K prompt
        dict(name="attn prefill 8K", op="attn", seqs=1, rows=2048, ctx_lo=8192, ctx_hi=8192, heads=128, topk=2048, page=64, pad=0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["plan", "append", "read", "attn", "attn", "attn"])
    page = rng.choice([64, 64, 128])
    if op == "plan":
        seqs = _log(rng, 1, 4096)
        hi = rng.choice([1, 2, _log(rng, 2, max(3, min(8192, 120000 // seqs)))])
        ctx = _log(rng, 64, 16384 if seqs > 512 else 131072)
        return dict(op=op, seqs=seqs, lo=rng.choice([0, 1]), hi=hi, ctx=ctx, page=rng.choice([16, 48, 64, 128]),
                    pad=_log(rng, 1, 1024), free=_log(rng, 8, 4096), release=rng.choice([0.0, 0.05, 0.2]))
    if op == "append":
        n = _log(rng, 1, 65536)
        return dict(op=op, n=n, tokens=_log(rng, n + 1, 131072), page=page)
    if op == "read":
        n = _log(rng, 1, 131072)
        return dict(op=op, n=n, tokens=_log(rng, 4096, 262144), page=page, holes=rng.choice([0, 1, n // 9]))
    heads = rng.choice([16, 32, 64, 128, 128])
    topk = rng.choice([2048, _log(rng, 16, 2048)])
    paged = rng.choice([0, page])
    if rng.random() < 0.3:                                       # a chunk of a prompt
        rows = _log(rng, 16, 2000)
        ctx = rows + _log(rng, 1, 14000)
        return dict(op=op, seqs=1, rows=rows, ctx_lo=ctx, ctx_hi=ctx, heads=heads, topk=topk, page=paged, pad=rng.choice([0, 5]))
    seqs, rows = _log(rng, 1, 64), rng.choice([1, 1, 2, 4])
    hi = _log(rng, 64, min(131072, 2000000 // seqs))
    return dict(op=op, seqs=seqs, rows=rows, ctx_lo=rng.randint(1, hi), ctx_hi=hi, heads=heads, topk=topk, page=paged, pad=rng.choice([0, 0, 3]))


# ---------------------------------------------------------------------------- inputs

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _latents(n, g):
    """Latent rows as a normalised down-projection gives them: unit scale, with a
    spread of magnitudes between channels; RoPE keys of unit scale."""
    x = torch.randn((n, D_C + D_R), device=DEV, generator=g)
    x[:, :D_C] *= 0.5 + torch.linspace(0, 1.5, D_C, device=DEV)[torch.arange(D_C, device=DEV) * 37 % D_C]
    return x.to(torch.bfloat16)


def _cache(tokens, g):
    """A cache of `tokens` packed latent rows, as earlier appends left it."""
    c = torch.empty((tokens, ROW), dtype=torch.uint8, device=DEV)
    for a in range(0, tokens, 131072):
        b = min(tokens, a + 131072)
        c[a:b] = _pack(_latents(b - a, g))
    return c


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    if op == "plan":
        return _prepare_plan(case, g)
    if op == "attn":
        return _prepare_attn(case, g)
    page, n = case["page"], case["n"]
    tokens = -(-case["tokens"] // page) * page
    s = dict(case, num_tokens=tokens)
    perm = torch.randperm(tokens // page, device=DEV, generator=g)
    pos = torch.arange(min(n, tokens), device=DEV)
    slots = perm[pos // page] * page + pos % page                # consecutive positions in scattered pages
    if op == "append":
        s["slot"] = slots
        s["k_new"] = torch.randn((n, D_IDX), device=DEV, generator=g)
        s["latent_new"] = _latents(n, g)
        s["latent"] = torch.zeros((tokens, ROW), dtype=torch.uint8, device=DEV)
        s["idx_k"] = torch.zeros((tokens, D_IDX), dtype=torch.uint8, device=DEV)
        s["idx_k_scale"] = torch.zeros(tokens, device=DEV)
    else:
        if n > tokens:                                           # several readers of one prefix
            slots = slots[torch.arange(n, device=DEV) % tokens]
        if case["holes"]:
            slots = slots.clone()
            slots[torch.randperm(n, device=DEV, generator=g)[: case["holes"]]] = -1
        s["slot"] = slots
        s["latent"] = _cache(tokens, g)
        k = torch.randn((tokens, D_IDX), device=DEV, generator=g)
        codes, s["idx_k_scale"] = _e4m3(k)
        s["idx_k"] = codes.view(torch.uint8)
    s["k_out"] = torch.zeros((n, D_IDX), device=DEV)
    s["latent_out"] = torch.zeros((n, D_C + D_R), dtype=torch.bfloat16, device=DEV)
    return s


def _rows(case):
    """Rows a server sizes its step for: the mean number of new tokens and `pad` more
    (some steps have more tokens than fit)."""
    return -(-case["seqs"] * (case["lo"] + case["hi"]) // 2) + case["pad"]


def _prepare_plan(case, g):
    B, page = case["seqs"], case["page"]
    width = -(-(case["ctx"] + case["hi"]) // page)
    n_new = torch.randint(case["lo"], case["hi"] + 1, (B,), device=DEV, generator=g)
    ctx = torch.randint(0, case["ctx"] + 1, (B,), device=DEV, generator=g)
    rel = torch.rand(B, device=DEV, generator=g) < case["release"]
    n_new = torch.where(rel, 0, n_new)
    held = (ctx + page - 1) // page
    start = torch.cumsum(held, 0) - held
    total = held.sum()
    num_pages = B * (-(-case["ctx"] // page)) + case["free"]
    perm = torch.randperm(num_pages, device=DEV, generator=g).to(torch.int32)
    col = torch.arange(width, device=DEV)
    table = torch.where(col[None] < held[:, None], perm[(start[:, None] + col[None]).clamp(max=num_pages - 1)], -1)
    free = torch.full((num_pages,), -1, dtype=torch.int32, device=DEV)
    free[: case["free"]] = perm[total + torch.arange(case["free"], device=DEV)]
    M = _rows(case)
    i32 = dict(dtype=torch.int32, device=DEV)
    return dict(case, num_pages=num_pages, width=width, max_tokens=M, seq_len=ctx.to(torch.int32), n_new=n_new.to(torch.int32),
                release_flags=rel.to(torch.int32), block_table=table.to(torch.int32).contiguous(), free_pages=free,
                free_count=torch.full((1,), case["free"], **i32),
                out=dict(seq_len_out=torch.zeros(B, **i32), free_count_out=torch.zeros(1, **i32), tok_start=torch.zeros(B + 1, **i32),
                         row_seq=torch.zeros(M, **i32), row_klen=torch.zeros(M, **i32), tok_pos=torch.zeros(M, **i32),
                         slot=torch.zeros(M, dtype=torch.int64, device=DEV), totals=torch.zeros(4, **i32)))


def _prepare_attn(case, g):
    B, R, topk, H, page = case["seqs"], case["rows"], case["topk"], case["heads"], case["page"]
    ctx = torch.randint(case["ctx_lo"], case["ctx_hi"] + 1, (B,), device=DEV, generator=g)
    unit = page or 64
    held = (ctx + unit - 1) // unit
    start = torch.cumsum(held, 0) - held
    units = int(held.sum())
    tokens, hi = units * unit, int(ctx.max())
    T = B * R + case["pad"]
    row_seq = torch.arange(T, device=DEV).clamp(max=B * R - 1) // R
    klen = (ctx[row_seq] - (R - 1 - torch.arange(T, device=DEV) % R)).clamp(min=0)
    klen[B * R:] = 0                                             # rows behind the last sequence see nothing
    s = dict(case, num_rows=T, num_tokens=tokens, max_klen=hi, row_seq=row_seq.to(torch.int32), row_klen=klen.to(torch.int32))
    if page:
        width = int(held.max())
        perm = torch.randperm(units, device=DEV, generator=g).to(torch.int32)
        col = torch.arange(width, device=DEV)
        s["block_table"] = torch.where(col[None] < held[:, None], perm[(start[:, None] + col[None]).clamp(max=units - 1)], -1).to(torch.int32).contiguous()
    else:
        s["seq_start"] = (start * unit).to(torch.int32)
    # the selection: top-k of random scores, ascending, -1 behind the last
    k = min(topk, hi)
    score = torch.rand((T, hi), device=DEV, generator=g)
    score.masked_fill_(torch.arange(hi, device=DEV)[None] >= klen[:, None], -1.0)
    val, pos = score.topk(k, dim=1)
    pos = torch.where(val >= 0, pos, hi).sort(dim=1).values
    idx = torch.full((T, topk), -1, dtype=torch.int32, device=DEV)
    idx[:, :k] = torch.where(pos < hi, pos, -1)
    s["idx"] = idx
    s["latent"] = _cache(tokens, g)
    s["q"] = (torch.randn((T, H, D_C + D_R), device=DEV, generator=g) * 0.05).to(torch.bfloat16)
    s["out"] = torch.zeros((T, H, D_C), dtype=torch.bfloat16, device=DEV)
    s["lse"] = torch.zeros((T, H), device=DEV)
    return s


# ---------------------------------------------------------------------------- plain forms

def _decode_scale(code):
    return (code.to(torch.int16) << 7).view(torch.float16).float()


def _pack(x):
    """Packed rows of bf16 latent rows: scale = amax / 7 rounded to the scale's
    8 bits, code = the nearest integer of [-7, 7] to x / scale."""
    n = x.shape[0]
    v = x[:, :D_C].float().view(n, D_C // GROUP, GROUP)
    r = v.abs().amax(-1) / torch.full((), 7.0, device=x.device)
    m, e = torch.frexp(r)
    normal = ((e - 1 + 15) << 3) + (torch.round(m * 16).to(torch.int32) - 8)
    code = torch.where(e >= -13, normal, torch.round(r * 131072.0).to(torch.int32)).clamp(max=SCALE_MAX_CODE)
    sc = _decode_scale(code)[..., None]
    q = torch.where(sc > 0, torch.round(v / torch.where(sc > 0, sc, 1.0)).clamp(-7, 7), 0.0)
    nib = (q.to(torch.int32) & 15).view(n, D_C // 8, 4, 2).transpose(2, 3).reshape(n, D_C // 8, 4, 2)
    by = (nib[..., 0] | (nib[..., 1] << 4)).to(torch.uint8).view(n, D_C // 2)
    rope = x[:, D_C:].contiguous().view(torch.uint8).view(n, 2 * D_R)
    return torch.cat([by, rope, code.to(torch.uint8)], dim=1)


def _unpack(rows):
    """fp32 values [n, d_c + d_r] of packed rows [n, ROW]."""
    n = rows.shape[0]
    by = rows[:, : D_C // 2]
    nib = torch.stack([by & 15, by >> 4], -1).view(n, D_C // 8, 2, 4).transpose(2, 3).reshape(n, D_C // GROUP, GROUP)
    q = nib.to(torch.int8)
    q = torch.where(q > 7, q - 16, q).float()
    lat = (q * _decode_scale(rows[:, D_C // 2 + 2 * D_R:])[..., None]).view(n, D_C)
    rope = rows[:, D_C // 2: D_C // 2 + 2 * D_R].contiguous().view(torch.bfloat16).float()
    return torch.cat([lat, rope], dim=1)


def _e4m3(k):
    amax = k.abs().amax(-1)
    s = amax / torch.full((), 448.0, device=k.device)
    s = torch.where(s > 0, s, 1.0)
    return (k / s[:, None]).clamp(-448, 448).to(torch.float8_e4m3fn), s


def _plain_read(s):
    ok = s["slot"] >= 0
    at = s["slot"].clamp(min=0)
    k = s["idx_k"][at].view(torch.float8_e4m3fn).float() * s["idx_k_scale"][at][:, None]
    s["k_out"].copy_(torch.where(ok[:, None], k, s["k_out"]))
    s["latent_out"].copy_(torch.where(ok[:, None], _unpack(s["latent"][at]).to(torch.bfloat16), s["latent_out"]))
    return [s["k_out"], s["latent_out"]]


def _plain_append(s):
    codes, scale = _e4m3(s["k_new"])
    s["idx_k"][s["slot"]] = codes.view(torch.uint8)
    s["idx_k_scale"][s["slot"]] = scale
    s["latent"][s["slot"]] = _pack(s["latent_new"])
    return _plain_read(s)


def _plain_plan(s):
    B, W, P, M, page = s["seqs"], s["width"], s["num_pages"], s["max_tokens"], s["page"]
    L, Nn, rel = s["seq_len"].long(), s["n_new"].long(), s["release_flags"] > 0
    F = s["free_count"].long()
    held = (L + page - 1) // page
    give = torch.where(rel, held, 0)
    give_end = torch.cumsum(give, 0)
    have = F + give_end[-1:]
    fits = ~rel & (L + Nn <= W * page)
    N = torch.where(fits, Nn, 0)
    need = torch.where(fits, (L + N + page - 1) // page - held, 0)
    go = fits & ((need == 0) | (torch.cumsum(need, 0) <= have)) & ((N == 0) | (torch.cumsum(N, 0) <= M))
    N, need = torch.where(go, N, 0), torch.where(go, need, 0)
    tok_end, pg_end = torch.cumsum(N, 0), torch.cumsum(need, 0)
    tok_start, pg_start = tok_end - N, pg_end - need
    total, taken = tok_end[-1:], pg_end[-1:]
    table, free = s["block_table"], s["free_pages"]
    # the stack of free pages: the list, then the pages handed back in this step
    i = torch.arange(P, device=DEV)
    by = torch.searchsorted(give_end, i, right=True).clamp(max=B - 1)
    back = table[by, (i - (give_end - give)[by]).clamp(0, W - 1)]
    stack = torch.where(i < F, free, back[(i - F).clamp(min=0)])
    # new entries of the block table
    col = torch.arange(W, device=DEV)[None] - held[:, None]
    page_of = stack[(have - 1 - pg_start[:, None] - col).clamp(0, P - 1)]
    table = torch.where((col >= 0) & (col < need[:, None]), page_of, table)
    # tokens
    t = torch.arange(M, device=DEV)
    b = torch.searchsorted(tok_end, t, right=True)
    live = t < total
    last = torch.where(N > 0, torch.arange(B, device=DEV), 0).amax()
    b = torch.where(live, b.clamp(max=B - 1), last)
    pos = L[b] + t - tok_start[b]
    slot = table[b, torch.where(live, pos // page, 0)].long() * page + pos % page
    free_out = have - taken
    o = s["out"]
    o["seq_len_out"].copy_(torch.where(rel, 0, L + N))
    o["free_count_out"].copy_(free_out)
    o["tok_start"].copy_(torch.cat([tok_start, total]))
    o["row_seq"].copy_(b)
    o["row_klen"].copy_(torch.where(live, pos + 1, 0))
    o["tok_pos"].copy_(torch.where(live, pos, -1))
    o["slot"].copy_(torch.where(live, slot, -1))
    o["totals"].copy_(torch.cat([total, taken, (~rel & ~go & (Nn > 0)).sum()[None], give_end[-1:]]))
    s["block_table"].copy_(table)
    s["free_pages"].copy_(torch.where((i >= F) & (i < free_out), stack, free))
    return dict(o, block_table=s["block_table"], free_pages=s["free_pages"])


def _physical(s):
    """Cache rows of the selected keys, and which of them count."""
    idx = s["idx"].long()
    ok = (idx >= 0) & (idx < s["row_klen"].long()[:, None])
    i = torch.where(ok, idx, 0)
    if s["page"]:
        row = s["block_table"][s["row_seq"].long()[:, None], i // s["page"]].long() * s["page"] + i % s["page"]
    else:
        row = s["seq_start"].long()[s["row_seq"].long()][:, None] + i
    return torch.where(ok, row, 0), ok


def _plain_attn(s):
    row, ok = _physical(s)
    T, k = row.shape
    if T * k < s["num_tokens"]:
        kv = _unpack(s["latent"][row.view(-1)]).view(T, k, D_C + D_R)
    else:
        kv = _unpack(s["latent"])[row]
    z = torch.matmul(s["q"].float(), kv.transpose(1, 2)) * SM_SCALE
    z.masked_fill_(~ok[:, None], -math.inf)
    m = z.amax(-1, keepdim=True)
    m = torch.where(m > -math.inf, m, 0.0)
    p = torch.exp(z.sub_(m))
    l = p.sum(-1, keepdim=True)
    o = torch.matmul(p, kv[..., :D_C]) / torch.where(l > 0, l, 1.0)
    s["out"].copy_(o)
    s["lse"].copy_((m + torch.log(l)).squeeze(-1))
    return [s["out"], s["lse"]]


# ---------------------------------------------------------------------------- the library's calls

def _native(s):
    """The descriptors and the workspace that a program keeps beside its tensors."""
    from long_context_sparse_04_b200 import _native as N
    p = lambda x: None if x is None else x.data_ptr()  # noqa: E731
    h = s["native"] = dict(N=N)
    st = torch.cuda.current_stream().cuda_stream
    if s["op"] == "plan":
        o = s["out"]
        h["cache"] = N.dsa_cache(block_table=p(s["block_table"]), page_size=s["page"], max_pages_per_seq=s["width"],
                                 num_seqs=s["seqs"], num_tokens=s["num_pages"] * s["page"])
        h["plan"] = N.dsa_plan(seq_len=p(s["seq_len"]), n_new=p(s["n_new"]), release=p(s["release_flags"]), seq_len_out=p(o["seq_len_out"]),
                               free_count=p(s["free_count"]), free_count_out=p(o["free_count_out"]), free_pages=p(s["free_pages"]),
                               free_capacity=s["num_pages"], max_tokens=s["max_tokens"], tok_start=p(o["tok_start"]), row_seq=p(o["row_seq"]),
                               row_klen=p(o["row_klen"]), tok_pos=p(o["tok_pos"]), slot=p(o["slot"]), totals=p(o["totals"]))
        nbytes = N.dsa_workspace_size(None, None, N.DSA_OP_BATCH_PLAN)
    else:
        h["dims"] = N.dsa_dims(n_idx_heads=64, d_idx=D_IDX, n_heads=s.get("heads", 128), d_c=D_C, d_r=D_R, topk=s.get("topk", 2048),
                               idx_dtype=N.DSA_FP8_E4M3, mla_dtype=N.DSA_INT4, sm_scale=SM_SCALE, algo=N.DSA_ALGO_AUTO)
        bt, paged = s.get("block_table"), s.get("block_table") is not None
        h["cache"] = N.dsa_cache(latent=p(s["latent"]), idx_k=p(s.get("idx_k")), idx_k_scale=p(s.get("idx_k_scale")), seq_start=p(s.get("seq_start")),
                                 block_table=p(bt), page_size=s["page"] if paged else 0, max_pages_per_seq=bt.shape[1] if paged else 0,
                                 num_seqs=s.get("seqs", 1), num_tokens=s["num_tokens"])
        h["rows"] = None
        op = N.DSA_OP_CACHE_APPEND
        if s["op"] == "attn":
            h["rows"] = N.dsa_rows(num_rows=s["num_rows"], row_seq=p(s["row_seq"]), row_klen=p(s["row_klen"]), max_klen=s["max_klen"], q_group=1)
            op = N.DSA_OP_SPARSE_MLA
        nbytes = N.dsa_workspace_size(h["dims"], h["rows"], op)
    h["ws"] = torch.empty(nbytes, dtype=torch.uint8, device=DEV)
    h["ws_bytes"] = nbytes
    N.dsa_workspace_init(h["ws"].data_ptr(), nbytes, st)
    return h


def run(state):
    s, op = state, state["op"]
    if not own:
        return {"plan": _plain_plan, "append": _plain_append, "read": _plain_read, "attn": _plain_attn}[op](s)
    h = s.get("native") or _native(s)
    N, ws, nb = h["N"], h["ws"].data_ptr(), h["ws_bytes"]
    st = torch.cuda.current_stream().cuda_stream
    if op == "plan":
        N.dsa_batch_plan(h["cache"], h["plan"], ws, nb, st)
        return dict(s["out"], block_table=s["block_table"], free_pages=s["free_pages"])
    if op == "attn":
        N.dsa_sparse_mla_fwd(h["dims"], h["rows"], h["cache"], s["q"].data_ptr(), s["idx"].data_ptr(), s["out"].data_ptr(), s["lse"].data_ptr(), ws, nb, st)
        return [s["out"], s["lse"]]
    n, slot = s["n"], s["slot"].data_ptr()
    if op == "append":
        N.dsa_cache_append_slots(h["dims"], h["cache"], n, slot, s["k_new"].data_ptr(), s["latent_new"].data_ptr(), ws, nb, st)
    N.dsa_cache_read(h["dims"], h["cache"], n, slot, s["k_out"].data_ptr(), s["latent_out"].data_ptr(), ws, nb, st)
    return [s["k_out"], s["latent_out"]]


# ---------------------------------------------------------------------------- work and 64-bit values

def work(case):
    op = case["op"]
    if op == "plan":
        B, page = case["seqs"], case["page"]
        rows = _rows(case)
        tokens = (rows - case["pad"]) * (1 - case["release"])
        held = B * case["release"] * case["ctx"] / 2 / page
        pages = min(case["free"] + held, tokens / page)
        # lengths in and out, token starts, 20 bytes a token; new table entries and their pages, pages handed back
        return {"bytes": 20 * B + 20 * rows + 8 * (pages + held), "flops": 0}
    n = case["n"] if "n" in case else 0
    value, packed = 4 * D_IDX + 2 * (D_C + D_R), D_IDX + 4 + ROW
    if op == "append":
        return {"bytes": n * (8 + 2 * value + 2 * packed), "flops": 0}
    if op == "read":
        return {"bytes": 8 * n + (n - case["holes"]) * value + min(n - case["holes"], case["tokens"]) * packed, "flops": 0}
    H, R, seqs = case["heads"], case["rows"], case["seqs"]
    T, ctx = seqs * R + case["pad"], (case["ctx_lo"] + case["ctx_hi"]) / 2
    keys = seqs * R * min(case["topk"], max(1.0, ctx - (R - 1) / 2))
    cached = min(keys, seqs * ctx)
    return {"bytes": T * H * (2 * (2 * D_C + D_R) + 4) + 4 * T * case["topk"] + cached * ROW, "flops": 2 * keys * H * (2 * D_C + D_R)}


def _np_unpack(rows):
    """Packed rows as float64 values, nibble by nibble from the format's text."""
    rows = rows.astype(np.int64)
    word = sum(rows[:, i: D_C // 2: 4] << (8 * i) for i in range(4))
    lat = np.empty((rows.shape[0], D_C))
    for d in range(8):
        v = (word >> (4 * (d // 2) + 16 * (d % 2))) & 15
        lat[:, d::8] = np.where(v >= 8, v - 16, v)
    e, m = rows[:, D_C // 2 + 2 * D_R:] >> 3, rows[:, D_C // 2 + 2 * D_R:] & 7
    sc = np.where(e > 0, (8 + m) * 2.0 ** (e - 18.0), m * 2.0 ** -17)
    lat *= np.repeat(sc, GROUP, axis=1)
    ro = rows[:, D_C // 2: D_C // 2 + 2 * D_R]
    rope = ((ro[:, 0::2] | (ro[:, 1::2] << 8)) << 16).astype(np.uint32).view(np.float32)
    return np.concatenate([lat, rope.astype(np.float64)], axis=1)


def _np_e4m3(codes):
    c = codes.astype(np.int64)
    e, m = (c >> 3) & 15, c & 7
    v = np.where(e > 0, (8 + m) * 2.0 ** (e - 10.0), m * 2.0 ** -9)
    return np.where(c & 128, -v, v)


def _np_quantise(x):
    """float64 values of quantised latents: the scale's candidates are listed, and
    the nearest (ties to the even code) to the fp32 quotient amax / 7 is taken."""
    sc = np.array([(8 + (c & 7)) * 2.0 ** ((c >> 3) - 18) if c >> 3 else (c & 7) * 2.0 ** -17 for c in range(SCALE_MAX_CODE + 1)])
    v = x[:, :D_C].reshape(x.shape[0], -1, GROUP)
    r = (np.abs(v).max(-1) / np.float32(7)).astype(np.float64)
    hi = np.searchsorted(sc, r).clip(1, SCALE_MAX_CODE)
    up, down = sc[hi] - r, r - sc[hi - 1]
    code = np.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, hi - 1)
    s = sc[code]
    y = (v / np.where(s > 0, s, 1).astype(np.float32)[..., None]).astype(np.float64)
    q = np.where(s[..., None] > 0, np.clip(np.rint(y), -7, 7), 0)
    return np.concatenate([(q * s[..., None]).reshape(x.shape[0], D_C), x[:, D_C:]], axis=1)


def exact(case, seed):
    if case["op"] == "plan":
        return None                                              # whole numbers only
    s = prepare(case, seed)
    if case["op"] == "attn":
        return _exact_attn(s)
    slot = s["slot"].cpu().numpy()
    if case["op"] == "append":
        k = s["k_new"].cpu().numpy()
        sc = np.abs(k).max(-1) / np.float32(448)
        sc = np.where(sc > 0, sc, np.float32(1))
        y = (k / sc[:, None]).astype(np.float64)
        grid = np.unique(np.abs(_np_e4m3(np.arange(127))))       # 0 .. 448 in code order
        a = np.minimum(np.abs(y), 448)
        hi = np.searchsorted(grid, a).clip(1, 126)
        up, down = grid[hi] - a, a - grid[hi - 1]
        code = np.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, hi - 1)
        kv = np.copysign(grid[code], y) * sc[:, None].astype(np.float64)
        return [kv, _np_quantise(s["latent_new"].float().cpu().numpy())]
    ok = (slot >= 0)[:, None]
    at = torch.from_numpy(np.maximum(slot, 0)).to(DEV)
    k = _np_e4m3(s["idx_k"][at].cpu().numpy()) * s["idx_k_scale"][at].cpu().numpy().astype(np.float64)[:, None]
    return [np.where(ok, k, 0.0), np.where(ok, _np_unpack(s["latent"][at].cpu().numpy()), 0.0)]


def _exact_attn(s):
    """Row by row in float64 on the GPU, from the definition."""
    T, H, k = s["num_rows"], s["heads"], s["topk"]
    out = torch.zeros((T, H, D_C), dtype=torch.float64, device=DEV)
    lse = torch.full((T, H), -math.inf, dtype=torch.float64, device=DEV)
    by = torch.arange(256, device=DEV)
    sc_of = torch.where(by >> 3 > 0, (8 + (by & 7)).double() * 2.0 ** ((by >> 3).double() - 18), (by & 7).double() * 2.0 ** -17)
    shift = torch.tensor([0, 16, 4, 20, 8, 24, 12, 28], device=DEV)
    seq, klen = s["row_seq"].tolist(), s["row_klen"].tolist()
    starts = None if s["page"] else s["seq_start"].tolist()
    for t in range(T):
        pos = s["idx"][t]
        pos = pos[(pos >= 0) & (pos < klen[t])].long()
        if not pos.numel():
            continue
        row = s["block_table"][seq[t]][pos // s["page"]].long() * s["page"] + pos % s["page"] if s["page"] else starts[seq[t]] + pos
        raw = s["latent"][row]
        word = raw[:, : D_C // 2].contiguous().view(torch.int32).long()
        v = (word[..., None] >> shift) & 15
        v = (v - 16 * (v >> 3)).double().reshape(-1, D_C // GROUP, GROUP)
        c = (v * sc_of[raw[:, D_C // 2 + 2 * D_R:].long()][..., None]).reshape(-1, D_C)
        r = raw[:, D_C // 2: D_C // 2 + 2 * D_R].contiguous().view(torch.bfloat16).double()
        q = s["q"][t].double()
        z = (q[:, :D_C] @ c.T + q[:, D_C:] @ r.T) * SM_SCALE
        lse[t] = torch.logsumexp(z, -1)
        out[t] = torch.exp(z - lse[t][:, None]) @ c
    return [out, lse]

"""Cases of the serving operators around a paged KV cache.

Four operators: attention over whole packed prompts, attention of new tokens over
a q8_0 paged cache, reading a paged cache back into packed rows, and the
verification of drafted tokens.  ``run`` computes them in plain torch operations
(32 bits, or 64 where a value can sit next to a border), or, with ``own`` set, with
the library's entry points.
"""
import math
import random

import torch

own = False

_DTYPE = {"f16": torch.float16, "bf16": torch.bfloat16}
_BS = 16  # tokens of a cache block


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def listed():
    qwen = dict(heads=14, kv_heads=2, head_dim=64)  # the repository's workload geometry
    wide = dict(heads=32, kv_heads=8, head_dim=128)
    return [
        # a handful of short prompts arriving together: latency
        dict(name="prompt tiny f16", op="prompt", dtype="f16", lens="1,17,64,200", **qwen),
        # the prompts of one admission step, lognormal lengths
        dict(name="prompt packed bf16", op="prompt", dtype="bf16", seqs=16, median=768, sigma=1.0, max_len=4096,
             lens_seed=5, **qwen),
        # one long document, wider heads
        dict(name="prompt 8192 f16 d128", op="prompt", dtype="f16", lens="8192", **wide),
        # the drafted tokens of 32 running sequences, scored in one call
        dict(name="chunk drafts bf16", op="chunk", dtype="bf16", seqs=32, median=512, sigma=1.0, max_len=4096,
             span_min=2, span_max=8, chunk_len=0, prefixes="", lens_seed=2, **qwen),
        # a mixed step: 16 decode rows beside two 512-token prompt chunks
        dict(name="chunk mixed f16", op="chunk", dtype="f16", seqs=16, median=768, sigma=1.0, max_len=4096, span_min=1,
             span_max=1, chunk_len=512, prefixes="1500,3000", lens_seed=5, **qwen),
        # prompt chunks far into long contexts
        dict(name="chunk long bf16", op="chunk", dtype="bf16", seqs=0, median=1, sigma=0.0, max_len=1, span_min=1,
             span_max=1, chunk_len=1024, prefixes="7168,7000,6144,5001", lens_seed=1, **qwen),
        # a few short sequences leave the cache: latency
        dict(name="gather tiny f16", op="gather", dtype="f16", q8=False, lens="1,17,64,200", **qwen),
        # sequences swapped out of a 16-bit cache, wider heads
        dict(name="gather b32 bf16 d128", op="gather", dtype="bf16", q8=False, seqs=32, median=512, sigma=1.0,
             max_len=4096, lens_seed=2, **wide),
        # a whole running batch read back from the 8-bit cache
        dict(name="gather b256 q8_0 bf16", op="gather", dtype="bf16", q8=True, seqs=256, median=1024, sigma=1.2,
             max_len=8192, lens_seed=4, **qwen),
        # a few sequences with four drafted tokens each: latency
        dict(name="verify 4 seqs", op="verify", seqs=4, draft_min=4, draft_max=4, vocab=151936, proposals="probs",
             lens_seed=1),
        # the whole running batch, one to seven drafted tokens
        dict(name="verify b256", op="verify", seqs=256, draft_min=1, draft_max=7, vocab=151936, proposals="probs",
             lens_seed=4),
        # drafts looked up in the prompt (no draft distribution), an odd vocabulary, some sequences without drafts
        dict(name="verify lookup odd vocab", op="verify", seqs=33, draft_min=0, draft_max=5, vocab=50257,
             proposals="tokens", lens_seed=3),
    ]


def _log_uniform(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("prompt", "prompt", "chunk", "chunk", "gather", "verify"))
    seed = rng.randrange(1 << 20)
    if op == "verify":
        seqs = _log_uniform(rng, 1, 200)
        lo = rng.randint(0 if seqs >= 16 else 1, 3)  # some sequence has a draft
        return dict(op=op, seqs=seqs, draft_min=lo, draft_max=lo + rng.randint(1, 4),
                    vocab=_log_uniform(rng, 1000, 150000), proposals=rng.choice(("probs", "probs", "tokens")),
                    lens_seed=seed)
    dtype = rng.choice(("f16", "bf16"))
    narrow = rng.choice(((14, 2), (8, 8), (12, 4), (16, 2), (32, 2), (5, 1)))
    broad = rng.choice(((32, 8), (28, 4), (16, 2)))
    max_len = _log_uniform(rng, 64, 4096)
    case = dict(op=op, dtype=dtype, seqs=_log_uniform(rng, 1, 24), median=_log_uniform(rng, 16, 1024),
                sigma=round(rng.uniform(0.0, 1.2), 2), max_len=max_len, lens_seed=seed)
    heads, kv_heads = narrow
    head_dim = 64
    if op == "chunk":
        lo = rng.randint(1, 4)
        n = rng.randint(0, 3)
        case.update(span_min=lo, span_max=lo + rng.randint(0, 12), chunk_len=_log_uniform(rng, 16, 600) if n else 0,
                    prefixes=",".join(str(_log_uniform(rng, 1, 5000)) for _ in range(n)))
    else:
        if op == "gather":
            case["q8"] = rng.random() < 0.5
        if not case.get("q8") and rng.random() < 0.5:
            heads, kv_heads = broad
            head_dim = 128
    case.update(heads=heads, kv_heads=kv_heads, head_dim=head_dim)
    return case


def _lens(case):
    """Tokens of each sequence: written out, or lognormal from the case's own seed."""
    if "lens" in case:
        return [int(x) for x in case["lens"].split(",")]
    rng = random.Random(case["lens_seed"])
    return [min(case["max_len"], max(1, round(case["median"] * math.exp(case["sigma"] * rng.gauss(0, 1)))))
            for _ in range(case["seqs"])]


def _spans(case):
    """(new tokens, tokens in the cache with them) of each sequence of a chunk case."""
    rng = random.Random(case["lens_seed"] + 1)
    spans = [(n, max(n, L)) for L in _lens(case) for n in (rng.randint(case["span_min"], case["span_max"]),)]
    if case["prefixes"]:
        spans += [(case["chunk_len"], case["chunk_len"] + int(p)) for p in case["prefixes"].split(",")]
    return spans


def _drafts(case):
    rng = random.Random(case["lens_seed"])
    return [rng.randint(case["draft_min"], case["draft_max"]) for _ in range(case["seqs"])]


def _seen(n, L):
    """Keys that the n last of L tokens see together."""
    return n * (L - n) + n * (n + 1) // 2


def work(case):
    if case["op"] == "verify":
        # one row of the target per sequence, one of the drafts' distribution too
        rows = case["seqs"] * (2 if case["proposals"] == "probs" else 1)
        return {"bytes": 4 * rows * case["vocab"], "flops": rows * case["vocab"]}
    hq, hkv, d = case["heads"], case["kv_heads"], case["head_dim"]
    row = d + d // 16 if case["op"] == "chunk" or case.get("q8") else 2 * d  # bytes of a cached row
    if case["op"] == "gather":
        return {"bytes": sum(_lens(case)) * hkv * 2 * (row + 2 * d), "flops": 0}
    spans = _spans(case) if case["op"] == "chunk" else [(n, n) for n in _lens(case)]
    qo = 2 * 2 * hq * d * sum(n for n, _ in spans)
    return {"bytes": qo + 2 * hkv * row * sum(L for _, L in spans), "flops": 4 * d * hq * sum(_seen(n, L) for n, L in spans)}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _starts(lens):
    out = [0]
    for n in lens:
        out.append(out[-1] + n)
    return torch.tensor(out, dtype=torch.int32, device="cuda")


def _quantise(x):
    """q8_0: codes and an fp16 scale for each 32 elements of a row."""
    b = x.float().unflatten(-1, (-1, 32))
    d = b.abs().amax(-1, keepdim=True) / 127.0
    inv = torch.where(d > 0, 1.0 / d, torch.zeros_like(d))
    codes = (b * inv).round().clamp(-127, 127).to(torch.int8)
    return codes.flatten(-2), d.squeeze(-1).to(torch.float16)


def _cache(case, lens, gen, q8):
    """A pool that holds the sequences in blocks of random order, and its tables."""
    need = [-(-n // _BS) for n in lens]
    total = sum(need) + max(1, sum(need) // 10)
    order = torch.randperm(total, generator=gen, device="cuda").to(torch.int32)
    width = max(need)
    at = torch.arange(width, device="cuda")
    first = torch.tensor([sum(need[:i]) for i in range(len(need))], device="cuda")
    count = torch.tensor(need, device="cuda")
    ids = order[(first[:, None] + at).clamp(max=total - 1)]
    tables = torch.where(at < count[:, None], ids, torch.full_like(ids, -1))
    shape = (total, case["kv_heads"], _BS, case["head_dim"])
    k = torch.randn(shape, generator=gen, device="cuda").to(_DTYPE[case["dtype"]])
    v = torch.randn(shape, generator=gen, device="cuda").to(_DTYPE[case["dtype"]])
    if q8:
        (kc, ks), (vc, vs) = _quantise(k), _quantise(v)
        return dict(kc=kc, ks=ks, vc=vc, vs=vs, tables=tables.contiguous())
    return dict(k=k, v=v, tables=tables.contiguous())


def _verify_inputs(case, gen):
    counts = _drafts(case)
    n, s, vocab = sum(counts), len(counts), case["vocab"]
    start = _starts(counts)
    rows = torch.randn(n + s, vocab, generator=gen, device="cuda").mul_(3.0)
    first = torch.repeat_interleave(torch.arange(s, device="cuda"), torch.tensor(counts, device="cuda"))
    mine = torch.arange(n, device="cuda") + first  # the target row that judges each draft
    st = dict(start=start, accept=torch.rand(n, generator=gen, device="cuda"),
              sample=torch.rand(s, generator=gen, device="cuda"), draft_probs=None, max_draft=max(counts))
    if case["proposals"] == "probs":
        guess = rows[mine] + torch.randn(n, vocab, generator=gen, device="cuda")
        noise = torch.rand(n, vocab, generator=gen, device="cuda").clamp_(min=1e-20)
        st["drafts"] = (guess - noise.log_().neg_().log_()).argmax(-1).to(torch.int32)
        st["draft_probs"] = torch.softmax(guess, -1)
    else:
        st["drafts"] = rows[mine].argmax(-1).to(torch.int32)
    st["target_probs"] = torch.softmax(rows, -1)
    st["tokens"] = torch.empty(n + s, dtype=torch.int32, device="cuda")
    st["accepted"] = torch.empty(s, dtype=torch.int32, device="cuda")
    return st


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    if case["op"] == "verify":
        return {"op": "verify", **_verify_inputs(case, gen)}
    hq, hkv, d, dt = case["heads"], case["kv_heads"], case["head_dim"], _DTYPE[case["dtype"]]
    if case["op"] == "prompt":
        lens = _lens(case)
        t = sum(lens)
        # one projection's output: q, k and v are slices of its rows
        qkv = torch.randn(t, hq + 2 * hkv, d, generator=gen, device="cuda").to(dt)
        return dict(op="prompt", q=qkv[:, :hq], k=qkv[:, hq:hq + hkv], v=qkv[:, hq + hkv:], start=_starts(lens),
                    longest=max(lens), scale=d ** -0.5, out=torch.empty(t, hq, d, dtype=dt, device="cuda"))
    if case["op"] == "chunk":
        spans = _spans(case)
        t = sum(n for n, _ in spans)
        st = dict(op="chunk", **_cache(case, [L for _, L in spans], gen, True))
        st.update(q=torch.randn(t, hq, d, generator=gen, device="cuda").to(dt), start=_starts([n for n, _ in spans]),
                  context=torch.tensor([L for _, L in spans], dtype=torch.int32, device="cuda"),
                  longest_span=max(n for n, _ in spans), longest=max(L for _, L in spans), scale=d ** -0.5,
                  out=torch.empty(t, hq, d, dtype=dt, device="cuda"))
        return st
    lens = _lens(case)
    t = sum(lens)
    st = dict(op="gather", start=_starts(lens), longest=max(lens), **_cache(case, lens, gen, case["q8"]))
    st["k_out"] = torch.empty(t, hkv, d, dtype=dt, device="cuda")
    st["v_out"] = torch.empty(t, hkv, d, dtype=dt, device="cuda")
    return st


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------
def _attend(q, k, v, n, L, scale):
    """q [S, N, Hq, D] (n[s] rows in use), k and v [S, M, Hkv, D] (L[s] in use), 32 bits:
    the rows are the last n of L tokens, each sees the keys up to its own."""
    S, N, hq, d = q.shape
    M, hkv = k.shape[1], k.shape[2]
    pos = (L - n)[:, None] + torch.arange(N, device=q.device)
    see = torch.arange(M, device=q.device) <= pos[:, :, None]
    see = (see & (torch.arange(N, device=q.device) < n[:, None])[:, :, None])[:, None, None]
    qg = q.view(S, N, hkv, hq // hkv, d).permute(0, 2, 3, 1, 4)
    z = torch.matmul(qg, k.permute(0, 2, 3, 1)[:, :, None]).mul_(scale).masked_fill_(~see, -math.inf)
    top = z.amax(-1, keepdim=True)
    p = z.sub_(torch.where(top > -math.inf, top, torch.zeros_like(top))).exp_()
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p, v.permute(0, 2, 1, 3)[:, :, None]) / torch.where(total > 0, total, torch.ones_like(total))
    return o.permute(0, 3, 1, 2, 4).reshape(S, N, hq, d)


def _padded(start, width, rows):
    """Row numbers [S, width] of packed sequences, and which of them are in use."""
    at = torch.arange(width, device=start.device)
    first, n = start[:-1].long(), (start[1:] - start[:-1]).long()
    return (first[:, None] + at).clamp(max=rows - 1), at < n[:, None], n


def _prompt(st):
    q, k, v = st["q"], st["k"], st["v"]
    idx, used, n = _padded(st["start"], st["longest"], q.shape[0])
    o = _attend(q[idx].float(), k[idx].float(), v[idx].float(), n, n, st["scale"])
    return o[used].to(q.dtype)


def _values(codes, scales):
    return (codes.float().unflatten(-1, (-1, 32)) * scales.float()[..., None]).flatten(-2)


def _chunk(st):
    q, tables = st["q"], st["tables"].long()
    idx, used, n = _padded(st["start"], st["longest_span"], q.shape[0])
    at = torch.arange(st["longest"], device=q.device)
    blk, off = tables[:, at // _BS].clamp(min=0), at % _BS
    k = _values(st["kc"][blk, :, off], st["ks"][blk, :, off])
    v = _values(st["vc"][blk, :, off], st["vs"][blk, :, off])
    o = _attend(q[idx].float(), k, v, n, st["context"].long(), st["scale"])
    return o[used].to(q.dtype)


def _gather(st):
    start = st["start"].long()
    t = torch.arange(st["k_out"].shape[0], device=start.device)
    s = torch.searchsorted(start, t, right=True) - 1
    p = t - start[s]
    blk, off = st["tables"].long()[s, p // _BS], p % _BS
    if "kc" in st:
        k, v = _values(st["kc"][blk, :, off], st["ks"][blk, :, off]), _values(st["vc"][blk, :, off], st["vs"][blk, :, off])
        return k.to(st["k_out"].dtype), v.to(st["v_out"].dtype)
    return st["k"][blk, :, off], st["v"][blk, :, off]


def _verify(st):
    p, q, drafts = st["target_probs"], st["draft_probs"], st["drafts"].long()
    idx, used, n = _padded(st["start"], max(1, st["max_draft"]), max(1, drafts.shape[0]))
    seq = torch.arange(n.shape[0], device=p.device)
    tok = torch.where(used, drafts[idx], 0)
    px = p[(idx + seq[:, None]).clamp(max=p.shape[0] - 1), tok].double()
    qx = q[idx, tok].double() if q is not None else torch.ones_like(px)
    ok = used & (st["accept"][idx].double() * qx < px)
    took = ok.int().cumprod(-1).sum(-1)  # drafts accepted before the first rejection
    row = st["start"][:-1].long() + took
    w = p[row + seq].double()
    refused = took < n
    if q is not None:
        rest = (w - q[row.clamp(max=q.shape[0] - 1)].double()).clamp_(min=0)
    else:
        rest = w.scatter(-1, drafts[row.clamp(max=drafts.shape[0] - 1)][:, None], 0.0)
    rest = torch.where(rest.sum(-1, keepdim=True) > 0, rest, w)
    w = torch.where(refused[:, None], rest, w)
    cum = w.cumsum(-1)
    last = (cum <= st["sample"].double()[:, None] * cum[:, -1:]).sum(-1)
    # packed: the accepted drafts, the drawn token, then -1
    out = torch.full((p.shape[0],), -1, dtype=torch.int32, device=p.device)
    keep = used & (torch.arange(idx.shape[1], device=p.device) < took[:, None])
    out[(idx + seq[:, None])[keep]] = tok[keep].to(torch.int32)
    out[row + seq] = last.to(torch.int32)
    return out, took.to(torch.int32)


# ---------------------------------------------------------------------------
# the library's entry points
# ---------------------------------------------------------------------------
_workspaces = {}  # a serving process keeps one workspace for all its calls


def _workspace(head_dim):
    from paged_kv_decode_ns_gb300 import binding as nb
    if head_dim not in _workspaces:
        _workspaces[head_dim] = nb.alloc_span_workspace(head_dim)
    return _workspaces[head_dim]


def _run_own(st):
    from paged_kv_decode_ns_gb300 import binding as nb
    if st["op"] == "prompt":
        nb.ns_prompt_attn(st["q"], st["k"], st["v"], st["start"], st["scale"], st["out"],
                          _workspace(st["q"].shape[-1]))
        return st["out"]
    if st["op"] == "chunk":
        nb.ns_paged_attn_prefill_q8_0(st["q"], st["start"], st["kc"], st["ks"], st["vc"], st["vs"], st["tables"],
                                      st["context"], st["scale"], st["out"], _workspace(st["q"].shape[-1]))
        return st["out"]
    if st["op"] == "gather":
        if "kc" in st:
            nb.ns_kv_gather_q8_0(st["kc"], st["ks"], st["vc"], st["vs"], st["tables"], st["start"], st["k_out"],
                                 st["v_out"])
        else:
            nb.ns_kv_gather(st["k"], st["v"], st["tables"], st["start"], st["k_out"], st["v_out"])
        return st["k_out"], st["v_out"]
    nb.ns_verify_drafts(st["target_probs"], st["draft_probs"], st["drafts"], st["start"], st["accept"], st["sample"],
                        st["tokens"], st["accepted"])
    return st["tokens"], st["accepted"]


def run(state):
    if own:
        return _run_own(state)
    return {"prompt": _prompt, "chunk": _chunk, "gather": _gather, "verify": _verify}[state["op"]](state)


# ---------------------------------------------------------------------------
# the definitions in 64 bits, sequence by sequence
# ---------------------------------------------------------------------------
def _exact_rows(q, k, v, scale):
    """q [n, Hq, D], k and v [L, Hkv, D] in 64 bits, a head at a time."""
    n, hq, _ = q.shape
    L, hkv, _ = k.shape
    hidden = torch.ones(n, L, dtype=torch.bool, device=q.device).triu_(L - n + 1)
    out = torch.empty_like(q)
    for j in range(hq):
        z = (q[:, j] @ k[:, j * hkv // hq].T) * scale
        z[hidden] = -math.inf
        out[:, j] = torch.softmax(z, -1) @ v[:, j * hkv // hq]
    return out


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "verify":
        return _exact_verify(st)
    start = st["start"].tolist()
    if case["op"] == "prompt":
        q, k, v = st["q"].double(), st["k"].double(), st["v"].double()
        return torch.cat([_exact_rows(q[a:b], k[a:b], v[a:b], st["scale"]) for a, b in zip(start, start[1:])])
    rows = st["context"].tolist() if case["op"] == "chunk" else [b - a for a, b in zip(start, start[1:])]
    cached = []
    for s, L in enumerate(rows):
        ids = st["tables"][s, : -(-L // _BS)].long()
        pair = []
        for x in ("k", "v"):
            if x + "c" in st:
                c, d = st[x + "c"][ids].double(), st[x + "s"][ids].double()
                c = c * d.repeat_interleave(32, dim=-1)
            else:
                c = st[x][ids].double()
            pair.append(c.transpose(1, 2).reshape(-1, case["kv_heads"], case["head_dim"])[:L])
        cached.append(pair)
    if case["op"] == "gather":
        return torch.cat([k for k, _ in cached]), torch.cat([v for _, v in cached])
    q = st["q"].double()
    return torch.cat([_exact_rows(q[a:b], k, v, st["scale"]) for a, b, (k, v) in zip(start, start[1:], cached)])


def _exact_verify(st):
    p, q = st["target_probs"], st["draft_probs"]
    start, drafts = st["start"].tolist(), st["drafts"].tolist()
    accept, sample = st["accept"].tolist(), st["sample"].tolist()
    tokens, accepted = [], []
    for s, (a, b) in enumerate(zip(start, start[1:])):
        w, taken = p[b + s].double(), b - a
        for i in range(a, b):
            x = drafts[i]
            target = p[i + s].double()
            other = q[i].double() if q is not None else torch.zeros_like(target).index_fill_(0, torch.tensor([x], device=p.device), 1.0)
            if not accept[i] * float(other[x]) < float(target[x]):
                w, taken = torch.relu(target - other), i - a
                w = w if float(w.sum()) > 0 else target
                break
        cum = torch.cumsum(w, 0)
        drawn = int(torch.searchsorted(cum, sample[s] * cum[-1], right=True))
        tokens += drafts[a:a + taken] + [drawn] + [-1] * (b - a - taken)
        accepted.append(taken)
    return torch.tensor(tokens, dtype=torch.int32), torch.tensor(accepted, dtype=torch.int32)

"""Cases of the rotary append and of the 4-bit (q4_0) paged cache.

Four operators: new tokens' queries and keys rotated by their positions, with keys and
values appended to a paged cache on the way; decode attention over a q4_0 cache;
attention of query spans over it; reading it back into packed rows.  ``run`` computes
them in plain torch operations in 32 bits, or, with ``own`` set, with the library's
entry points.
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
    rope = dict(op="rope", rotary=64, interleaved=False, pad=0, first="0")
    return [
        # the new token of four running sequences, before a decode step: latency
        dict(rope, name="rope 4 tokens f16", dtype="f16", pool="16", lens="1,1,1,1", first="0,16,63,199", **qwen),
        # one long prompt into a 16-bit cache, wider heads; the rotated keys go to the prompt's attention too
        dict(rope, name="rope 8192 bf16 d128", dtype="bf16", pool="16", lens="8192", **{**wide, "rotary": 128}),
        # the prompts of one admission step into an 8-bit cache and read back from it, as for a swap-out
        dict(rope, name="rope q8_0 prompts bf16", dtype="bf16", pool="q8_0", seqs=16, median=768, sigma=1.0, max_len=4096,
             lens_seed=5, **qwen),
        # 512-token chunks of four prompts into a 4-bit cache and read back, half of the width rotated in pairs
        dict(rope, name="rope q4_0 chunks f16 d128", dtype="f16", pool="q4_0", lens="512,512,512,509",
             **{**wide, "interleaved": True, "first": "7168,2000,512,0"}),
        # a decode step of four short sequences: latency
        dict(name="decode tiny f16", op="decode", dtype="f16", lens="1,17,64,200", **qwen),
        # the decode step of a whole running batch
        dict(name="decode b256 bf16", op="decode", dtype="bf16", seqs=256, median=1024, sigma=1.2, max_len=8192,
             lens_seed=4, **qwen),
        # few long contexts
        dict(name="decode 8x4096 f16", op="decode", dtype="f16", lens=",".join(["4096"] * 8), **qwen),
        # very long documents of uneven lengths, wider heads
        dict(name="decode documents bf16 d128", op="decode", dtype="bf16", lens="131072,65536,20001,333", **wide),
        # the drafted tokens of 32 running sequences, scored in one call
        dict(name="chunk drafts bf16", op="chunk", dtype="bf16", seqs=32, median=512, sigma=1.0, max_len=4096,
             span_min=2, span_max=8, chunk_len=0, prefixes="", lens_seed=2, **qwen),
        # prompt chunks far into long contexts
        dict(name="chunk long f16", op="chunk", dtype="f16", seqs=0, median=1, sigma=0.0, max_len=1, span_min=1,
             span_max=1, chunk_len=1024, prefixes="7168,7000,6144,5001", lens_seed=1, **qwen),
        # a few short sequences leave the cache: latency
        dict(name="gather tiny bf16", op="gather", dtype="bf16", lens="1,17,64,200", **qwen),
        # sequences swapped out or read as a prefix, wider heads
        dict(name="gather b32 f16 d128", op="gather", dtype="f16", seqs=32, median=512, sigma=1.0, max_len=4096,
             lens_seed=2, **wide),
    ]


def _log_uniform(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("rope", "rope", "decode", "decode", "chunk", "gather"))
    dtype = rng.choice(("f16", "bf16"))
    narrow = rng.choice(((14, 2), (8, 8), (12, 4), (16, 2), (32, 2), (5, 1), (9, 1)))
    broad = rng.choice(((32, 8), (28, 4), (16, 2), (20, 2)))
    (heads, kv_heads), head_dim = (narrow, 64) if op == "chunk" or rng.random() < 0.6 else (broad, 128)
    case = dict(op=op, dtype=dtype, seqs=_log_uniform(rng, 1, 24), median=_log_uniform(rng, 16, 1024),
                sigma=round(rng.uniform(0.0, 1.2), 2), max_len=_log_uniform(rng, 64, 4096),
                lens_seed=rng.randrange(1 << 20), heads=heads, kv_heads=kv_heads, head_dim=head_dim)
    if op == "rope":
        pool = rng.choice(("16", "q8_0", "q4_0") if head_dim == 64 else ("16", "q4_0"))
        if rng.random() < 0.4:  # a decode step's tokens instead of prompts
            case.update(seqs=_log_uniform(rng, 1, 300), median=1, sigma=0.0, max_len=1)
        case.update(pool=pool, rotary=16 * rng.randint(1, head_dim // 16), interleaved=rng.random() < 0.4,
                    pad=rng.choice((0, 0, 1, 5, 24)) if pool == "16" else 0,
                    first=",".join(str(_log_uniform(rng, 1, 20000) - 1) for _ in range(case["seqs"])))
    elif op == "decode":
        if rng.random() < 0.3:  # long contexts
            case.update(seqs=rng.randint(1, 4), median=_log_uniform(rng, 4000, 40000), max_len=60000, sigma=0.4)
        else:
            case.update(seqs=_log_uniform(rng, 1, 200))
    elif op == "chunk":
        lo = rng.randint(1, 4)
        n = rng.randint(0, 3)
        case.update(span_min=lo, span_max=lo + rng.randint(0, 12), chunk_len=_log_uniform(rng, 16, 600) if n else 0,
                    prefixes=",".join(str(_log_uniform(rng, 1, 5000)) for _ in range(n)))
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


def _first(case):
    """Position of each sequence's first new token."""
    at = [int(x) for x in case["first"].split(",")]
    n = len(_lens(case))
    return at if len(at) == n else at * n


def _seen(n, L):
    """Keys that the n last of L tokens see together."""
    return n * (L - n) + n * (n + 1) // 2


def work(case):
    hq, hkv, d = case["heads"], case["kv_heads"], case["head_dim"]
    q4 = d // 2 + d // 16  # bytes of a cached row: codes and scales
    if case["op"] == "rope":
        t = sum(_lens(case))
        row = {"16": 2 * d, "q8_0": d + d // 16, "q4_0": q4}[case["pool"]]
        table = len({p for f, n in zip(_first(case), _lens(case)) for p in range(f, f + n)}) * case["rotary"] * 4
        moved = t * (2 * (hq + 2 * hkv) * d + 12 + 2 * hq * d + 2 * hkv * row) + table
        # the rotated keys besides the 16-bit cache; the rows read back from the others
        moved += t * 2 * hkv * d if case["pool"] == "16" else t * 2 * hkv * (row + 2 * d)
        return {"bytes": moved, "flops": 3 * t * (hq + hkv) * case["rotary"]}
    if case["op"] == "gather":
        return {"bytes": sum(_lens(case)) * hkv * 2 * (q4 + 2 * d), "flops": 0}
    spans = _spans(case) if case["op"] == "chunk" else [(1, n) for n in _lens(case)]
    qo = 2 * 2 * hq * d * sum(n for n, _ in spans)
    return {"bytes": qo + 2 * hkv * q4 * sum(L for _, L in spans), "flops": 4 * d * hq * sum(_seen(n, L) for n, L in spans)}


# ---------------------------------------------------------------------------
# the cache's formats: codes and an fp16 scale for each 32 elements of a row
# ---------------------------------------------------------------------------
def _quantise_q8_0(x):
    b = x.unflatten(-1, (-1, 32))
    d = b.abs().amax(-1, keepdim=True) / 127.0
    inv = torch.where(d > 0, 1.0 / d, torch.zeros_like(d))
    codes = (b * inv).round().clamp(-127, 127).to(torch.int8)
    return codes.flatten(-2), d.squeeze(-1).clamp(max=65504.0).to(torch.float16)


def _quantise_q4_0(x):
    """The element of largest magnitude becomes code 0 (-8 steps); byte j of a row holds element 2j in
    its low half and 2j + 1 in its high half."""
    b = x.unflatten(-1, (-1, 32))
    top, low = b.amax(-1, keepdim=True), b.amin(-1, keepdim=True)
    d = torch.where(top >= -low, top, low) * -0.125
    scale = d.clamp(-65504.0, 65504.0).to(torch.float16)
    inv = torch.where(scale != 0, 1.0 / d, torch.zeros_like(d))
    codes = (b * inv + 8.5).floor().clamp(0, 15).to(torch.uint8).flatten(-2)
    return codes[..., 0::2] | (codes[..., 1::2] << 4), scale.squeeze(-1)


def _values_q8_0(codes, scales):
    return (codes.float().unflatten(-1, (-1, 32)) * scales.float()[..., None]).flatten(-2)


def _values_q4_0(codes, scales):
    c = torch.stack((codes & 15, codes >> 4), -1).flatten(-2).float() - 8.0
    return (c.unflatten(-1, (-1, 32)) * scales.float()[..., None]).flatten(-2)


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _starts(lens):
    out = [0]
    for n in lens:
        out.append(out[-1] + n)
    return torch.tensor(out, dtype=torch.int32, device="cuda")


def _tables(lens, gen):
    """Blocks in random order for sequences of these lengths: (blocks of the pool, their table)."""
    need = [-(-n // _BS) for n in lens]
    total = sum(need) + max(1, sum(need) // 10)
    order = torch.randperm(total, generator=gen, device="cuda").to(torch.int32)
    at = torch.arange(max(need), device="cuda")
    first = torch.tensor([sum(need[:i]) for i in range(len(need))], device="cuda")
    count = torch.tensor(need, device="cuda")
    ids = order[(first[:, None] + at).clamp(max=total - 1)]
    return total, torch.where(at < count[:, None], ids, torch.full_like(ids, -1)).contiguous()


def _normal(shape, gen, dtype):
    return torch.randn(shape, generator=gen, device="cuda").to(dtype)


def _rope_inputs(case, gen):
    hq, hkv, d, dt, r = case["heads"], case["kv_heads"], case["head_dim"], _DTYPE[case["dtype"]], case["rotary"]
    lens, first = _lens(case), _first(case)
    t, pad = sum(lens), case["pad"]
    seq = torch.repeat_interleave(torch.arange(len(lens), device="cuda"), torch.tensor(lens, device="cuda"))
    start = _starts(lens)
    within = torch.arange(t, device="cuda") - start[:-1].long()[seq]
    # the new tokens lie in blocks of their own, from each sequence's first entry on
    total, tables = _tables(lens, gen)
    slots = tables.long()[seq, within // _BS] * _BS + within % _BS
    positions = torch.tensor(first, device="cuda")[seq] + within
    # rows behind the last token, as a captured step of a fixed size has them
    slots = torch.cat((slots, torch.full((pad,), -1, device="cuda", dtype=torch.int64)))
    positions = torch.cat((positions, torch.zeros(pad, device="cuda", dtype=torch.int64))).to(torch.int32)
    # cosines and sines of every position up to the last, angles in 64 bits
    angle = torch.arange(max(f + n for f, n in zip(first, lens)), device="cuda", dtype=torch.float64)[:, None] \
        * 10000.0 ** (-torch.arange(0, r, 2, device="cuda", dtype=torch.float64) / r)
    qkv = _normal((t + pad, hq + 2 * hkv, d), gen, dt)  # one projection's output: q, k and v are slices of its rows
    st = dict(op="rope", pool=case["pool"], interleaved=case["interleaved"], q=qkv[:, :hq], k=qkv[:, hq:hq + hkv],
              v=qkv[:, hq + hkv:], positions=positions, slots=slots, start=start, tables=tables,
              cos_sin=torch.cat((angle.cos(), angle.sin()), -1).float(),
              q_out=torch.zeros(t + pad, hq, d, dtype=dt, device="cuda"))
    rows = (total, hkv, _BS)
    if case["pool"] == "16":
        st.update(k_pool=_normal(rows + (d,), gen, dt), v_pool=_normal(rows + (d,), gen, dt),
                  k_out=torch.zeros(t + pad, hkv, d, dtype=dt, device="cuda"))
    else:
        width, code = (d, torch.int8) if case["pool"] == "q8_0" else (d // 2, torch.uint8)
        for x in ("k", "v"):
            st[x + "c"] = torch.zeros(rows + (width,), dtype=code, device="cuda")
            st[x + "s"] = torch.zeros(rows + (d // 32,), dtype=torch.float16, device="cuda")
            st[x + "_rows"] = torch.empty(t, hkv, d, dtype=dt, device="cuda")
    return st


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    if case["op"] == "rope":
        return _rope_inputs(case, gen)
    hq, hkv, d, dt = case["heads"], case["kv_heads"], case["head_dim"], _DTYPE[case["dtype"]]
    spans = _spans(case) if case["op"] == "chunk" else [(1, n) for n in _lens(case)]
    lens = [L for _, L in spans]
    total, tables = _tables(lens, gen)
    st = dict(op=case["op"], tables=tables, longest=max(lens), scale=d ** -0.5)
    for x in ("k", "v"):
        st[x + "c"], st[x + "s"] = _quantise_q4_0(_normal((total, hkv, _BS, d), gen, dt).float())
    if case["op"] == "gather":
        st["start"] = _starts(lens)
        for x in ("k", "v"):
            st[x + "_rows"] = torch.empty(sum(lens), hkv, d, dtype=dt, device="cuda")
        return st
    rows = sum(n for n, _ in spans)
    st.update(q=_normal((rows, hq, d), gen, dt), context=torch.tensor(lens, dtype=torch.int32, device="cuda"),
              out=torch.empty(rows, hq, d, dtype=dt, device="cuda"), start=_starts([n for n, _ in spans]),
              longest_span=max(n for n, _ in spans))
    return st


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------
def _rotate(x, cos, sin, interleaved):
    """x [T, H, D] in 32 bits, cos and sin [T, r / 2]."""
    half = cos.shape[-1]
    c, s = cos[:, None], sin[:, None]
    a, b = (x[..., 0:2 * half:2], x[..., 1:2 * half:2]) if interleaved else (x[..., :half], x[..., half:2 * half])
    ra, rb = a * c - b * s, b * c + a * s
    y = x.clone()
    if interleaved:
        y[..., 0:2 * half:2], y[..., 1:2 * half:2] = ra, rb
    else:
        y[..., :half], y[..., half:2 * half] = ra, rb
    return y


def _rope(st):
    half = st["cos_sin"].shape[-1] // 2
    table = st["cos_sin"][st["positions"].long()]
    q = _rotate(st["q"].float(), table[:, :half], table[:, half:], st["interleaved"])
    k = _rotate(st["k"].float(), table[:, :half], table[:, half:], st["interleaved"])
    on = st["slots"] >= 0
    blk, off = st["slots"][on] // _BS, st["slots"][on] % _BS
    st["q_out"][on] = q.to(st["q_out"].dtype)[on]
    if st["pool"] == "16":
        st["k_out"][on] = k.to(st["k_out"].dtype)[on]
        st["k_pool"][blk, :, off] = st["k_out"][on]
        st["v_pool"][blk, :, off] = st["v"][on]
        return st["q_out"], st["k_out"], st["k_pool"], st["v_pool"]
    quantise, values = (_quantise_q8_0, _values_q8_0) if st["pool"] == "q8_0" else (_quantise_q4_0, _values_q4_0)
    rows = []
    for x, full in (("k", k), ("v", st["v"].float())):
        codes, scales = quantise(full[on])
        st[x + "c"][blk, :, off], st[x + "s"][blk, :, off] = codes, scales
        rows.append(values(st[x + "c"][blk, :, off], st[x + "s"][blk, :, off]).to(st["q_out"].dtype))
    return st["q_out"], rows[0], rows[1]


def _attend(st):
    """The rows of q are the last n of L tokens of each sequence; each sees the keys up to its own."""
    q, tables = st["q"], st["tables"].long()
    _, hq, d = q.shape
    hkv = st["kc"].shape[1]
    first, n = st["start"][:-1].long(), (st["start"][1:] - st["start"][:-1]).long()
    span = torch.arange(st["longest_span"], device=q.device)
    idx, used = (first[:, None] + span).clamp(max=q.shape[0] - 1), span < n[:, None]
    at = torch.arange(st["longest"], device=q.device)
    blk, off = tables[:, at // _BS].clamp(min=0), at % _BS
    k = _values_q4_0(st["kc"][blk, :, off], st["ks"][blk, :, off])
    pos = (st["context"].long() - n)[:, None] + span
    see = ((at <= pos[:, :, None]) & used[:, :, None])[:, None, None]
    qg = q[idx].float().view(len(n), -1, hkv, hq // hkv, d).permute(0, 2, 3, 1, 4)
    z = torch.matmul(qg, k.permute(0, 2, 3, 1)[:, :, None]).mul_(st["scale"]).masked_fill_(~see, -math.inf)
    del k
    top = z.amax(-1, keepdim=True)
    p = z.sub_(torch.where(top > -math.inf, top, torch.zeros_like(top))).exp_()
    total = p.sum(-1, keepdim=True)
    v = _values_q4_0(st["vc"][blk, :, off], st["vs"][blk, :, off])
    o = torch.matmul(p, v.permute(0, 2, 1, 3)[:, :, None]) / torch.where(total > 0, total, torch.ones_like(total))
    return o.permute(0, 3, 1, 2, 4).reshape(len(n), -1, hq, d)[used].to(q.dtype)


def _gather(st):
    start = st["start"].long()
    t = torch.arange(st["k_rows"].shape[0], device=start.device)
    s = torch.searchsorted(start, t, right=True) - 1
    p = t - start[s]
    blk, off = st["tables"].long()[s, p // _BS], p % _BS
    return tuple(_values_q4_0(st[x + "c"][blk, :, off], st[x + "s"][blk, :, off]).to(st["k_rows"].dtype) for x in "kv")


# ---------------------------------------------------------------------------
# the library's entry points
# ---------------------------------------------------------------------------
_workspaces = {}  # a serving process keeps its workspaces for all its calls


def _workspace(st):
    from paged_kv_decode_ns_gb300 import binding as nb
    rows, hq, d = st["q"].shape
    hkv = st["kc"].shape[1]
    key = ("span", d) if st["op"] == "chunk" else (rows, hq, hkv, d)
    if key not in _workspaces:
        _workspaces[key] = nb.alloc_span_workspace(d) if st["op"] == "chunk" else nb.alloc_workspace(rows, hq, hkv, d)
    return _workspaces[key]


def _run_own(st):
    from paged_kv_decode_ns_gb300 import binding as nb
    if st["op"] == "rope":
        head = (st["q"], st["k"], st["v"], st["positions"], st["cos_sin"], st["slots"], st["q_out"])
        if st["pool"] == "16":
            nb.ns_rope_kv_append(*head, st["k_pool"], st["v_pool"], k_out=st["k_out"], interleaved=st["interleaved"])
            return st["q_out"], st["k_out"], st["k_pool"], st["v_pool"]
        pools = (st["kc"], st["ks"], st["vc"], st["vs"])
        append, gather = (nb.ns_rope_kv_append_q8_0, nb.ns_kv_gather_q8_0) if st["pool"] == "q8_0" else \
            (nb.ns_rope_kv_append_q4_0, nb.ns_kv_gather_q4_0)
        append(*head, *pools, interleaved=st["interleaved"])
        gather(*pools, st["tables"], st["start"], st["k_rows"], st["v_rows"])
        return st["q_out"], st["k_rows"], st["v_rows"]
    pools = (st["kc"], st["ks"], st["vc"], st["vs"])
    if st["op"] == "gather":
        nb.ns_kv_gather_q4_0(*pools, st["tables"], st["start"], st["k_rows"], st["v_rows"])
        return st["k_rows"], st["v_rows"]
    if st["op"] == "decode":
        nb.ns_paged_attn_decode_q4_0(st["q"], *pools, st["tables"], st["context"], st["scale"], st["out"], _workspace(st))
    else:
        nb.ns_paged_attn_prefill_q4_0(st["q"], st["start"], *pools, st["tables"], st["context"], st["scale"], st["out"],
                                      _workspace(st))
    return st["out"]


def run(state):
    if own:
        return _run_own(state)
    return {"rope": _rope, "decode": _attend, "chunk": _attend, "gather": _gather}[state["op"]](state)


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------
def _exact_values(codes, scales):
    """Elements of q4_0 rows: step times (code - 8)."""
    out = torch.empty(codes.shape[:-1] + (2 * codes.shape[-1],), dtype=torch.float64, device=codes.device)
    out[..., 0::2] = (codes % 16).double() - 8.0
    out[..., 1::2] = torch.div(codes, 16, rounding_mode="floor").double() - 8.0
    return out * scales.double().repeat_interleave(32, dim=-1)


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


def _to32(x):
    """What 32 bits hold of a value in 64 (one rounding): the formats decide their codes in 32 bits."""
    return x.float().double()


def _exact_turned(x, table, interleaved, in_steps):
    """Each pair of x as a complex number times the position's; `in_steps`: with the products and
    the sum rounded to 32 bits, as the 8- and 4-bit formats see them."""
    half = table.shape[-1] // 2
    c, s = table[:, None, :half].double(), table[:, None, half:].double()
    fit = _to32 if in_steps else (lambda y: y)
    out = x.double()
    i = torch.arange(half, device=x.device)
    re, im = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
    a, b = out[..., re], out[..., im]
    out[..., re] = fit(fit(a * c) - fit(b * s))
    out[..., im] = fit(fit(a * s) + fit(b * c))
    return out


def _exact_held(x, pool):
    """What the 8- or 4-bit cache holds of x [T, H, D]: its rules, each step in 64 bits rounded to 32."""
    b = x.reshape(*x.shape[:-1], -1, 32)
    if pool == "q8_0":
        d = _to32(b.abs().amax(-1) / 127)
        codes = torch.round(_to32(b * _to32(1 / d)[..., None])).clamp(-127, 127)
    else:
        m = b.gather(-1, b.abs().argmax(-1, keepdim=True)).squeeze(-1)
        m = torch.where((b == m.abs()[..., None]).any(-1), m.abs(), m)  # of +a and -a the positive one
        d = m / -8
        codes = torch.floor(_to32(_to32(b * _to32(1 / d)[..., None]) + 8.5)).clamp(max=15) - 8
    return (codes * d.half().double()[..., None]).reshape(x.shape)


def _exact_rope(st):
    table = st["cos_sin"][st["positions"].long()]
    on = st["slots"] >= 0
    q = _exact_turned(st["q"], table, st["interleaved"], False)
    q[~on] = 0.0  # rows without a token stay as they were
    if st["pool"] != "16":
        k = _exact_turned(st["k"], table, st["interleaved"], True)
        return q, _exact_held(k, st["pool"]), _exact_held(st["v"].double(), st["pool"])
    k = _exact_turned(st["k"], table, st["interleaved"], False)
    k[~on] = 0.0
    pools = []
    for pool, rows in ((st["k_pool"], k), (st["v_pool"], st["v"].double())):
        flat = pool.double().transpose(1, 2).reshape(-1, *rows.shape[1:])
        flat[st["slots"][on]] = rows[on]
        pools.append(flat.reshape(pool.shape[0], _BS, *rows.shape[1:]).transpose(1, 2))
    return q, k, pools[0], pools[1]


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "rope":
        return _exact_rope(st)
    start = st["start"].tolist()
    rows = [b - a for a, b in zip(start, start[1:])] if case["op"] == "gather" else st["context"].tolist()
    cached = []
    for s, L in enumerate(rows):
        ids = st["tables"][s, : -(-L // _BS)].long()
        cached.append([_exact_values(st[x + "c"][ids], st[x + "s"][ids]).transpose(1, 2)
                       .reshape(-1, case["kv_heads"], case["head_dim"])[:L] for x in "kv"])
    if case["op"] == "gather":
        return torch.cat([k for k, _ in cached]), torch.cat([v for _, v in cached])
    q = st["q"].double()
    return torch.cat([_exact_rows(q[a:b], k, v, st["scale"]) for a, b, (k, v) in zip(start, start[1:], cached)])

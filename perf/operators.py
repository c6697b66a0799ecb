"""The serving operators beside the step compile, as cases that can be timed:

* ``attention``  the step's query tokens (single tokens, chunks, or both) attend
                 to their requests' pages: causal, with an optional tanh cap on
                 the scores, a sliding window, a linear bias by distance and a
                 prefix that every query of its request sees;
* ``logprobs``   log probabilities of given tokens with their rank, the row's
                 entropy and the top alternatives;
* ``copy`` / ``move``  pages copied in every layer's caches (forks), and pages
                 moved with every block-table entry that names them (compaction).

``run`` computes a case in elementary torch operations, or, with ``own`` true,
through ``ragged_input_compilation_amd``."""
import math

import numpy as np
import torch

own = False

_DT = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}


# ---- cases ----------------------------------------------------------------------

def _attn(name, kind, reqs, shape, heads, kv_heads, dim, block, dtype, lo, hi, chunk=1, chunks=0, cap=0.0, window=0,
          alibi=False, prefix=False):
    """``reqs`` requests; ``chunks`` of them compute up to ``chunk`` new tokens
    (kind "chunk": all lengths drawn; "fixed": exactly ``chunk``), the others
    one; cached lengths U[lo, hi].  ``shape`` seeds the lengths."""
    return {"name": name, "op": "attention", "kind": kind, "reqs": reqs, "shape": shape, "heads": heads,
            "kv_heads": kv_heads, "dim": dim, "block": block, "dtype": dtype, "lo": lo, "hi": hi, "chunk": chunk,
            "chunks": chunks, "cap": cap, "window": window, "alibi": alibi, "prefix": prefix}


def _logp(name, rows, vocab, dtype, top):
    return {"name": name, "op": "logprobs", "rows": rows, "vocab": vocab, "dtype": dtype, "top": top}


def _pages(name, op, pages, pool, layers, block, row, reqs=0, per_req=0):
    return {"name": name, "op": op, "pages": pages, "pool": pool, "layers": layers, "block": block, "row": row,
            "reqs": reqs, "per_req": per_req}


def listed():
    return [
        # a handful of requests, one of them in the middle of its prompt: latency counts
        _attn("attention_few", "chunk", 3, 1, 4, 2, 64, 16, "f16", 0, 24, chunk=12, chunks=2),
        # one user's decode over a long history: few rows, a long axis
        _attn("attention_decode_one", "decode", 1, 2, 32, 8, 128, 16, "bf16", 60001, 60001),
        # 256 decodes with contexts U[128, 4096], the decode-heavy configuration's layer
        _attn("attention_decode_heavy", "decode", 256, 3, 32, 8, 128, 16, "bf16", 128, 4096),
        # decodes of a model with capped scores and a sliding window, heads of 64, odd lengths
        _attn("attention_decode_window", "decode", 97, 4, 16, 8, 64, 16, "f16", 511, 8191, cap=50.0, window=1024),
        # decodes and chunks in one step, the mixed configuration's proportions
        _attn("attention_mixed", "chunk", 124, 5, 32, 8, 128, 16, "bf16", 256, 8192, chunk=2048, chunks=4),
        # long chunks over long cached prefixes in 64-token pages
        _attn("attention_long_chunk", "fixed", 4, 6, 32, 8, 128, 64, "bf16", 0, 30720, chunk=2048, chunks=4),
        # prompts with a fully visible prefix and a bias by distance
        _attn("attention_prefix_bias", "chunk", 9, 7, 16, 16, 64, 16, "bf16", 0, 700, chunk=1500, chunks=9, alibi=True,
              prefix=True),
        # the sampled token of one request
        _logp("logprobs_one", 1, 32000, "f32", 5),
        # every row of a decode step
        _logp("logprobs_decode", 256, 128256, "bf16", 20),
        # a prompt scored token by token
        _logp("logprobs_prompt", 2048, 152064, "bf16", 5),
        # forked samples: the partly filled page of each is copied in 32 layers
        _pages("copy_fork", "copy", 24, 512, 32, 16, 2048),
        # a pool compacted: pages move in 4 layers and 1024 block tables follow
        _pages("move_compact", "move", 1500, 8000, 4, 16, 2048, reqs=1024, per_req=6),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    while True:
        case = _draw(rng)
        w = work(case)
        if w["flops"] <= 2.0e12 and w["bytes"] <= 2.2e9:         # at most the largest listed case
            return case


def _draw(rng):
    what = rng.choice(["attention", "attention", "attention", "logprobs", "pages"])
    if what == "attention":
        kind = rng.choice(["decode", "decode", "chunk", "fixed"])
        kv_heads = rng.choice([1, 2, 4, 8])
        heads = kv_heads * rng.choice([1, 2, 4, 8] if kv_heads < 8 else [1, 2, 4])
        reqs = _log_int(rng, 1, 256) if kind == "decode" else _log_int(rng, 1, 40)
        hi = _log_int(rng, 16, 4096 if reqs > 16 else 30000)
        chunks = 0 if kind == "decode" else rng.randint(1, min(reqs, 8))
        chunk = 1 if kind == "decode" else _log_int(rng, 2, 2048)
        return _attn("", kind, reqs, rng.randrange(1 << 30), heads, kv_heads, rng.choice([64, 128]),
                     rng.choice([16, 16, 32, 64, 24]), rng.choice(["f16", "bf16"]), rng.randint(0, hi), hi, chunk=chunk,
                     chunks=chunks, cap=rng.choice([0.0, 0.0, 30.0]), window=rng.choice([0, 0, _log_int(rng, 8, 4096)]),
                     alibi=rng.random() < 0.25, prefix=kind != "decode" and rng.random() < 0.25)
    if what == "logprobs":
        vocab = _log_int(rng, 1000, 152064)
        rows = _log_int(rng, 1, 2048)
        return _logp("", rows, vocab, rng.choice(["f16", "bf16", "f32"]) if rows <= 1000 else "bf16",
                     rng.choice([0, 1, 5, 20]))
    layers = rng.choice([1, 4, 8])
    block = rng.choice([16, 32, 24])
    row = rng.choice([256, 512, 1024, 2048])
    if rng.random() < 0.5:
        pages = _log_int(rng, 1, 600)
        return _pages("", "copy", pages, 2 * pages + rng.randint(2, 400), layers, block, row)
    reqs = _log_int(rng, 1, 300)
    per = rng.randint(1, 8)
    used = reqs * per + 1
    return _pages("", "move", rng.randint(1, max(1, min(500, used // 2))), 2 * used + 8, layers, block, row, reqs=reqs,
                  per_req=per)


# ---- attention -------------------------------------------------------------------

def _lengths(case):
    """Query and total lengths of each request, from the case alone."""
    r = np.random.default_rng(case["shape"])
    n = case["reqs"]
    c = r.integers(case["lo"], case["hi"] + 1, n)
    q = np.ones(n, np.int64)
    which = r.permutation(n)[:case["chunks"]]
    q[which] = case["chunk"] if case["kind"] == "fixed" else r.integers(1, case["chunk"] + 1, len(which))
    prefix = r.integers(0, c + q + 1) if case["prefix"] else np.zeros(n, np.int64)
    return q, c + q, prefix


def _slopes(case):
    return [2.0 ** (-8.0 * (h + 1) / case["heads"]) for h in range(case["heads"])]


def _visible(case):
    """Number of (query, key) pairs and of key rows that any query sees."""
    q, total, prefix = _lengths(case)
    pairs = rows = 0
    for n, t, pre in zip(q.tolist(), total.tolist(), prefix.tolist()):
        p = np.arange(t - n, t, dtype=np.int64)
        end = np.maximum(p + 1, pre)
        lo = np.maximum(p + 1 - case["window"], 0) if case["window"] else np.zeros_like(p)
        pairs += int((end - lo).sum())
        rows += int(end.max() - lo.min())
    return pairs, rows


def _prepare_attention(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = _DT[case["dtype"]]
    q_len, total, prefix = _lengths(case)
    B, D = case["block"], case["dim"]
    nb = -(-total // B)
    pool = int(nb.sum()) + 9
    n = int(q_len.sum())
    rand = lambda *s: torch.randn(s, generator=g, device="cuda", dtype=torch.float32).to(dt)
    ids = (torch.randperm(pool - 1, generator=g, device="cuda")[:int(nb.sum())] + 1).to(torch.int32).cpu().numpy()
    table = np.zeros((case["reqs"], int(nb.max())), np.int32)
    at = 0
    for i, k in enumerate(nb.tolist()):
        table[i, :k] = ids[at:at + k]
        at += k
    i32 = lambda a: torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()
    st = {"case": case, "q": rand(n, case["heads"], D) * 1.5, "kc": rand(pool, B, case["kv_heads"], D),
          "vc": rand(pool, B, case["kv_heads"], D), "table": i32(table), "q_len": q_len.tolist(),
          "total": total.tolist(), "prefix": prefix.tolist(), "qsl": i32(np.concatenate([[0], np.cumsum(q_len)])),
          "seq": i32(total), "scale": D ** -0.5, "max_q": int(q_len.max()), "max_seq": int(total.max()),
          "slopes": torch.tensor(_slopes(case), device="cuda") if case["alibi"] else None,
          "prefix_dev": i32(prefix) if case["prefix"] else None}
    if own:
        from ragged_input_compilation_amd import runner
        st["out"] = torch.empty_like(st["q"])
        st["workspace"] = runner.attention_workspace(st["q"], st["kc"], case["reqs"], st["max_q"], st["max_seq"])
    return st


def _attention_plain(st):
    case = st["case"]
    H, KH, D = case["heads"], case["kv_heads"], case["dim"]
    G = H // KH
    out = torch.empty_like(st["q"])
    start = 0
    for i, (n, t, pre) in enumerate(zip(st["q_len"], st["total"], st["prefix"])):
        blocks = st["table"][i, :-(-t // case["block"])].long()
        k = st["kc"][blocks].reshape(-1, KH, D)[:t].permute(1, 2, 0).float().contiguous()     # [KH, D, t]
        v = st["vc"][blocks].reshape(-1, KH, D)[:t].permute(1, 0, 2).float().contiguous()     # [KH, t, D]
        j = torch.arange(t, device="cuda")
        step = max(1, (1 << 28) // (H * t))
        for a in range(0, n, step):
            b = min(n, a + step)
            q = st["q"][start + a:start + b].float().reshape(b - a, KH, G, D).permute(1, 2, 0, 3)
            s = torch.matmul(q.reshape(KH, G * (b - a), D).contiguous(), k).view(KH, G, b - a, t) * st["scale"]
            if case["cap"]:
                s = case["cap"] * torch.tanh(s / case["cap"])
            p = torch.arange(t - n + a, t - n + b, device="cuda")[:, None]
            if case["alibi"]:
                s = s - st["slopes"].view(KH, G, 1, 1) * (p - j).abs().float()
            see = (j <= p) | (j < pre)
            if case["window"]:
                see = see & (p - j < case["window"])
            s = s.masked_fill(~see, float("-inf"))
            e = torch.exp(s - s.amax(dim=-1, keepdim=True))
            o = torch.matmul(e.view(KH, G * (b - a), t), v).view(KH, G, b - a, D) / e.sum(dim=-1, keepdim=True)
            out[start + a:start + b] = o.permute(2, 0, 1, 3).reshape(b - a, H, D).to(out.dtype)
        start += n
    return out


def _attention_own(st):
    from ragged_input_compilation_amd import runner
    case = st["case"]
    runner.paged_attention(st["q"], st["kc"], st["vc"], st["table"], st["qsl"], st["seq"], st["max_q"], st["max_seq"],
                           st["out"], scale=st["scale"], softcap=case["cap"], window=case["window"],
                           alibi_slopes=st["slopes"], prefix_lens=st["prefix_dev"], workspace=st["workspace"])
    return st["out"]


def _attention_exact(st):
    """Head by head in float64: weights exp(score - logsumexp) over the keys
    of each request in logical order."""
    case = st["case"]
    G = case["heads"] // case["kv_heads"]
    out = torch.zeros(st["q"].shape, dtype=torch.float64, device="cuda")
    first = 0
    for i in range(case["reqs"]):
        n, t = st["q_len"][i], st["total"][i]
        tok = torch.arange(t, device="cuda")
        page, off = st["table"][i].long()[tok // case["block"]], tok % case["block"]
        pos = torch.arange(t - n, t, device="cuda").unsqueeze(1)
        hidden = (tok > pos) & (tok >= st["prefix"][i])
        if case["window"]:
            hidden |= tok <= pos - case["window"]
        for h in range(case["heads"]):
            kh = st["kc"][page, off, h // G].double()
            vh = st["vc"][page, off, h // G].double()
            for a in range(0, n, 1024):
                b = min(n, a + 1024)
                score = st["q"][first + a:first + b, h].double().mm(kh.t()) * float(st["scale"])
                if case["cap"]:
                    score = torch.tanh(score / case["cap"]) * case["cap"]
                if case["alibi"]:
                    score -= st["slopes"][h].double() * (pos[a:b] - tok).abs()
                score[hidden[a:b]] = -math.inf
                out[first + a:first + b, h] = torch.exp(score - torch.logsumexp(score, 1, keepdim=True)).mm(vh)
        first += n
    return out


# ---- log probabilities -------------------------------------------------------------

def _prepare_logprobs(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rows, V = case["rows"], case["vocab"]
    logits = torch.empty((rows, V), dtype=_DT[case["dtype"]], device="cuda")
    targets = torch.empty(rows, dtype=torch.int32, device="cuda")
    for a in range(0, rows, 256):
        b = min(rows, a + 256)
        x = (torch.randn((b - a, V), generator=g, device="cuda") * 2.5).to(logits.dtype)
        # a few likely continuations stand out of the bulk
        hot = torch.randint(0, V, (b - a, 8), generator=g, device="cuda")
        x.scatter_(1, hot, (torch.rand((b - a, 8), generator=g, device="cuda") * 12 + 4).to(x.dtype))
        logits[a:b] = x
        # targets sampled from the distribution itself
        u = torch.rand((b - a, V), generator=g, device="cuda").clamp_min_(1e-20)
        targets[a:b] = (x.float() - torch.log(-torch.log(u))).argmax(dim=1).to(torch.int32)
    st = {"case": case, "logits": logits, "targets": targets}
    if own:
        from ragged_input_compilation_amd import runner
        st["out"] = runner.alloc_logprobs(rows, V, case["top"])
    return st


def _logprobs_plain(st):
    top, rows = st["case"]["top"], st["case"]["rows"]
    V = st["case"]["vocab"]
    lp, ent, rank, ids, tlp = [], [], [], [], []
    idx = torch.arange(V, device="cuda")
    for a in range(0, rows, 128):
        x = st["logits"][a:a + 128].float()
        t = st["targets"][a:a + 128].long()[:, None]
        m = x.amax(dim=1, keepdim=True)
        d = x - m
        e = torch.exp(d)
        total = e.sum(dim=1, keepdim=True)
        lse = torch.log(total)
        xt = x.gather(1, t)
        lp.append((xt - m - lse)[:, 0])
        ent.append((lse - (e * d).sum(dim=1, keepdim=True) / total)[:, 0])
        rank.append((1 + (x > xt).sum(dim=1) + ((x == xt) & (idx < t)).sum(dim=1)).to(torch.int32))
        # order by value, then by the lower token id
        bits = (x + 0.0).view(torch.int32).long()
        key = torch.where(bits < 0, -1 - (bits & 0x7FFFFFFF), bits) * V + (V - 1 - idx)
        best = V - 1 - key.topk(top, dim=1).values.remainder(V) if top else key[:, :0]
        ids.append(best.to(torch.int32))
        tlp.append(x.gather(1, best) - m - lse)
    return tuple(torch.cat(z) for z in (lp, rank, ent, ids, tlp))


def _logprobs_own(st):
    from ragged_input_compilation_amd import runner
    o = runner.token_logprobs(st["logits"], st["targets"], st["case"]["top"], st["out"])
    return o.logprob, o.rank, o.entropy, o.top_ids, o.top_logprobs


def _logprobs_exact(st):
    top, rows = st["case"]["top"], st["case"]["rows"]
    res = []
    for r in range(0, rows, 64):
        x = st["logits"][r:r + 64].double()
        t = st["targets"][r:r + 64].long()
        logp = x - torch.logsumexp(x, dim=1, keepdim=True)
        n = torch.arange(x.shape[0], device="cuda")
        order = torch.sort(x, dim=1, descending=True, stable=True).indices
        place = (order == t[:, None]).nonzero()[:, 1] + 1
        best = order[:, :top]
        res.append((logp[n, t], place.to(torch.int32), -(logp.exp() * logp).sum(dim=1), best.to(torch.int32),
                    logp.gather(1, best)))
    return tuple(torch.cat(z) for z in zip(*res))


# ---- pages ----------------------------------------------------------------------

def _prepare_pages(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = np.random.default_rng(seed)
    pool, n = case["pool"], case["pages"]
    shape = (pool, case["block"], case["row"] // 2)
    caches = []
    for _ in range(2 * case["layers"]):
        bits = torch.randint(-32768, 32768, shape, generator=g, device="cuda", dtype=torch.int16)
        caches.append((bits & 0x3FFF).view(torch.bfloat16))          # finite values
    st = {"case": case, "kc": caches[::2], "vc": caches[1::2]}
    tables = []
    if case["op"] == "copy":
        ids = r.permutation(np.arange(1, pool))[:2 * n]
        src, dst = ids[:n], ids[n:]
    else:
        # live pages are scattered over the pool; the highest move into the lowest free ones
        used = r.permutation(np.arange(1, pool))[:case["reqs"] * case["per_req"]]
        at = 0
        for _ in range(case["reqs"]):
            k = int(r.integers(1, case["per_req"] + 1))
            tables.append(used[at:at + k].astype(np.int32))
            at += k
        live = np.sort(used[:at])
        free = np.setdiff1d(np.arange(1, pool), live)
        n = min(n, len(live), len(free))
        src, dst = live[::-1][:n], free[:n]
        st["table"] = torch.zeros((case["reqs"], case["per_req"]), dtype=torch.int32, device="cuda")
        host = np.zeros((case["reqs"], case["per_req"]), np.int32)
        for i, ids in enumerate(tables):
            host[i, :len(ids)] = ids
        st["table"].copy_(torch.from_numpy(host))
    st["src"], st["dst"] = np.ascontiguousarray(src, np.int32), np.ascontiguousarray(dst, np.int32)
    if own:
        from ragged_input_compilation_amd import _ric as ric, runner
        per = max(case["per_req"], 1)
        b = runner.Batch(ric.make_config(max_num_reqs=max(case["reqs"], 1), max_model_len=per * case["block"],
                                         block_size=case["block"], max_blocks_per_req=per, max_num_batched_tokens=64,
                                         num_kv_blocks=pool, null_block=0, staging_bytes=0))
        b.block_table().zero_()
        for i, ids in enumerate(tables):
            ric.ric_add_request(b.h, i, [1], 1, 0, ids)
        ric.ric_flush(b.h)
        st["batch"] = b
    return st


def _bits(st):
    """The caches as whole numbers: copies keep every bit."""
    return [c.view(torch.int16) for c in st["kc"] + st["vc"]]


def _pages_plain(st):
    src, dst = torch.from_numpy(st["src"]).cuda().long(), torch.from_numpy(st["dst"]).cuda().long()
    for c in st["kc"] + st["vc"]:
        c[dst] = c[src]
    outs = _bits(st)
    if st["case"]["op"] == "move":
        to = torch.arange(st["case"]["pool"], dtype=torch.int32, device="cuda")
        to[src] = dst.to(torch.int32)
        st["table"] = to[st["table"].long()]
        outs.append(st["table"])
    return outs


def _pages_own(st):
    from ragged_input_compilation_amd import runner
    b = st["batch"]
    if st["case"]["op"] == "copy":
        runner.copy_blocks(b, st["src"], st["dst"], st["kc"], st["vc"])
        return _bits(st)
    runner.move_blocks(b, st["src"], st["dst"], st["kc"], st["vc"])
    return _bits(st) + [b.block_table()[:st["case"]["reqs"], :st["case"]["per_req"]]]


# ---- the interface ----------------------------------------------------------------

def prepare(case, seed):
    make = {"attention": _prepare_attention, "logprobs": _prepare_logprobs}.get(case["op"], _prepare_pages)
    return make(case, seed)


def run(state):
    op = state["case"]["op"]
    if op == "attention":
        return _attention_own(state) if own else _attention_plain(state)
    if op == "logprobs":
        return _logprobs_own(state) if own else _logprobs_plain(state)
    return _pages_own(state) if own else _pages_plain(state)


def work(case):
    if case["op"] == "attention":
        pairs, rows = _visible(case)
        q = int(_lengths(case)[0].sum())
        per = case["dim"] * 2
        return {"bytes": 2 * q * case["heads"] * per + 2 * rows * case["kv_heads"] * per,
                "flops": 4 * pairs * case["heads"] * case["dim"]}
    if case["op"] == "logprobs":
        size = 4 if case["dtype"] == "f32" else 2
        n = case["rows"] * case["vocab"]
        return {"bytes": n * size + case["rows"] * (16 + 8 * case["top"]), "flops": 4 * n}
    moved = 2 * case["pages"] * case["layers"] * case["block"] * case["row"]
    return {"bytes": 2 * moved + 8 * case["reqs"] * case["per_req"], "flops": 0}


def exact(case, seed):
    if case["op"] not in ("attention", "logprobs"):
        return None
    global own
    was, own = own, False
    try:
        state = prepare(case, seed)
    finally:
        own = was
    return _attention_exact(state) if case["op"] == "attention" else _logprobs_exact(state)

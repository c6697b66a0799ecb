"""Definitions in 64 bits of the operators around the step, and seeded inputs
for their tests.  Nothing here calls the library."""
import numpy as np
import torch

HALF_STEP = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


def attention_inputs(lens, *, heads, kv_heads, dim, block, dtype, seed=0, extra_blocks=3, pad_tokens=0, device="cuda",
                     unused=float("nan"), scale_q=1.0):
    """``lens``: (query tokens, total length) per request.  Pages in a seeded
    order; every cache row that belongs to no request holds ``unused``."""
    g = torch.Generator().manual_seed(seed)
    nb = [max(0, -(-t // block)) for _, t in lens]
    pool = sum(nb) + extra_blocks
    order = torch.randperm(pool, generator=g)
    width = max([1] + nb)
    table = torch.full((len(lens), width), -7, dtype=torch.int32)      # entries past a row's pages name no page
    kc = torch.full((pool, block, kv_heads, dim), unused)
    vc = torch.full((pool, block, kv_heads, dim), unused)
    at = 0
    for i, (_, t) in enumerate(lens):
        ids = order[at:at + nb[i]]
        at += nb[i]
        table[i, :nb[i]] = ids.to(torch.int32)
        for j in range(0, t, block):
            m = min(block, t - j)
            kc[ids[j // block], :m] = torch.randn((m, kv_heads, dim), generator=g)
            vc[ids[j // block], :m] = torch.randn((m, kv_heads, dim), generator=g)
    n = sum(q for q, _ in lens)
    q = torch.randn((n + pad_tokens, heads, dim), generator=g) * scale_q
    qsl = np.concatenate([[0], np.cumsum([a for a, _ in lens])]).astype(np.int32)
    return dict(q=q.to(dtype).to(device), kc=kc.to(dtype).to(device), vc=vc.to(dtype).to(device),
                table=table.to(device), qsl=torch.from_numpy(qsl).to(device),
                seq=torch.tensor([t for _, t in lens], dtype=torch.int32, device=device), lens=list(lens))


def attention_reference(inp, *, scale, softcap=0.0, window=0, slopes=None, prefix=None, bad_blocks=()):
    """(out, tolerance) in float64, rows of the requests in order.

    The tolerance adds what each rounding can do.  A = sum p|v| / sum p bounds
    the output.  (1) Weights p in (0, 1] rounded to the type's bits, half a
    step each: half * A, and for float16 below its normals 2^-25 each.  (2) The
    output's own rounding: half * |out|.  (3) A score off by ds changes every
    weight by at most e^ds: 4 ds A covers numerator and denominator; ds is the
    float32 dot product's bound (dim + 8) 2^-24 sum|q||k| scale and 2^-21 of the
    scores' and biases' size (scale, cap, bias, max and exp each round once or
    twice).  (4) Float32 sums over n keys: (n + 64) 2^-24 A."""
    q, kc, vc = inp["q"], inp["kc"], inp["vc"]
    dt = q.dtype
    half = HALF_STEP[dt]
    H, D = q.shape[1:]
    KH, B = kc.shape[2], kc.shape[1]
    G = H // KH
    dev = q.device
    outs, tols = [], []
    start = 0
    for i, (n, t) in enumerate(inp["lens"]):
        qi = q[start:start + n].double()
        start += n
        out = torch.zeros((n, H, D), dtype=torch.float64, device=dev)
        tol = torch.zeros_like(out)
        outs.append(out)
        tols.append(tol)
        if n == 0 or t <= 0:
            continue
        j = torch.arange(t, device=dev)
        ids = inp["table"][i].long()[torch.div(j, B, rounding_mode="floor").clamp(max=inp["table"].shape[1] - 1)]
        ok = (ids >= 0) & (ids < kc.shape[0]) & (j < inp["table"].shape[1] * B)
        for x in bad_blocks:
            ok &= ids != x
        ids = ids.clamp(0, kc.shape[0] - 1)
        k, v = kc[ids, j % B].double(), vc[ids, j % B].double()
        pos = torch.arange(t - n, t, device=dev)[:, None]
        see = (j <= pos)
        if prefix is not None:
            see = see | (j < prefix[i])
        if window:
            see = see & (j > pos - window)
        see = see & ok
        for h in range(H):
            kk, vv = k[:, h // G], v[:, h // G]
            s = (qi[:, h] @ torch.nan_to_num(kk, nan=0.0, posinf=0.0, neginf=0.0).T) * scale
            mag = qi[:, h].abs() @ torch.nan_to_num(kk, nan=0.0, posinf=0.0, neginf=0.0).abs().T * abs(scale)
            if not torch.isfinite(kk).all():           # non-finite keys: the rows that see them, element by element
                bad = ~torch.isfinite(kk).all(dim=1)
                s[:, bad] = (qi[:, h][:, None, :] * kk[bad][None]).sum(-1) * scale
            if softcap:
                s = softcap * torch.tanh(s / softcap)
            bias = torch.zeros_like(s) if slopes is None else float(slopes[h]) * (pos - j).abs().double()
            s = (s - bias).masked_fill(~see, float("-inf"))
            m = s.amax(dim=1, keepdim=True)
            live = m.squeeze(1) > float("-inf")
            live |= m.squeeze(1).isnan()
            p = torch.exp(s - m)
            p = torch.where(see, p, torch.zeros_like(p))
            l = p.sum(dim=1, keepdim=True)
            good = torch.isfinite(vv)
            v0 = torch.where(good, vv, torch.zeros_like(vv))
            o = (p @ v0) / l
            a = (p @ v0.abs()) / l
            hit = (see.double() @ (~good).double()) > 0        # a visible value is not finite
            o = torch.where(hit, torch.full_like(o, float("nan")), o)
            near = see & (s > m - 40)
            big = lambda x: torch.where(near, x, torch.zeros_like(x)).amax(dim=1, keepdim=True)
            ds = (D + 8) * 2.0 ** -24 * big(mag) + 2.0 ** -21 * (big(s.abs().nan_to_num(0.0, 0.0, 0.0)) + big(bias))
            e = half * a + half * o.abs() + 4 * ds * a + (t + 64) * 2.0 ** -24 * a
            if dt == torch.float16:
                e = e + see.sum(1, keepdim=True) * 2.0 ** -25 * v0.abs().amax(dim=0, keepdim=True) / l + 2.0 ** -25
            out[:, h] = torch.where(live[:, None], o, torch.zeros_like(o))
            tol[:, h] = torch.where(live[:, None], e, torch.zeros_like(e))
    cat = lambda x: torch.cat(x) if x else torch.zeros((0, H, D), dtype=torch.float64, device=dev)
    return cat(outs), cat(tols)


def check_attention(got, want, tol, label=""):
    got = got.double()
    fin = torch.isfinite(want)
    assert not torch.isfinite(got[~fin]).any(), f"{label}: finite where a visible value is not"
    err = (got - want).abs()
    bad = fin & ~(err <= tol)
    if bad.any():
        k = tuple(int(x) for x in bad.nonzero()[0])
        raise AssertionError(f"{label}: {int(bad.sum())} of {bad.numel()} outside; first {k}: got {got[k].item():.6g} "
                             f"want {want[k].item():.6g} tolerance {tol[k].item():.3g}")


def logprob_reference(x, targets, top_k):
    """(logprob, rank, entropy, top_ids, top_logprobs) of float64 rows x, NaN
    ordered first, then by value, ties by the lower id."""
    x = x.double()
    rows, V = x.shape
    m = x.amax(dim=1, keepdim=True)
    none = (m == float("-inf"))
    d = x - torch.where(none, torch.zeros_like(m), m)
    e = torch.exp(d)
    S = e.sum(dim=1, keepdim=True)
    lp = torch.where(none, torch.full_like(d, float("-inf")), d - torch.log(S))
    ent = torch.log(S) - torch.where(e > 0, e * d, torch.zeros_like(d)).sum(dim=1, keepdim=True) / S
    ent = torch.where(none, torch.zeros_like(ent), ent)
    broken = x.isnan().any(dim=1, keepdim=True) | (x == float("inf")).any(dim=1, keepdim=True)
    lp = torch.where(broken, torch.full_like(lp, float("nan")), lp)
    ent = torch.where(broken, torch.full_like(ent, float("nan")), ent)
    order = torch.sort(torch.where(x.isnan(), torch.full_like(x, float("inf")), x) , dim=1, descending=True,
                       stable=True).indices
    # a NaN lies above +inf
    first = x.isnan().gather(1, order).to(torch.int8)
    order = order.gather(1, torch.sort(first, dim=1, descending=True, stable=True).indices)
    place = torch.empty_like(order)
    place.scatter_(1, order, torch.arange(V, device=x.device).expand(rows, V).contiguous())
    has = (targets >= 0) & (targets < V)
    t = targets.long().clamp(0, V - 1)[:, None]
    z = torch.zeros(rows, dtype=torch.float64, device=x.device)
    logprob = torch.where(has, lp.gather(1, t)[:, 0], z)
    rank = torch.where(has, place.gather(1, t)[:, 0] + 1, torch.zeros_like(place[:, 0]))
    ids = order[:, :top_k]
    return logprob, rank, ent[:, 0], ids, lp.gather(1, ids)

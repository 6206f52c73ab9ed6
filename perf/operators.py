"""What the cache and window operators are measured on: their inputs, their plain forms and their values in 64 bits.

Five operators that a server of a hybrid sparse-attention model runs around the selection layers:

  token_write / token_read   one layer's K/V rows into (and out of) the e4m3 cache with one scale per token that the
                             decode layers read: scale = max|x|/448 (1 for a row of zeros), code = e4m3(x / scale)
  paged_write / paged_read   the same for a paged cache with one power-of-two scale per page of tokens and KV head
  paged_decode               one query token per sequence over that paged cache, all of it or a window and the first
                             tokens (sinks)
  window_attn                causal attention of a chunk of a prompt to a window of recent tokens and the sinks

`own` False: plain torch in 32 bits.  `own` True: this repository's kernels."""
import math

import torch

own = False

E4M3_MAX = 448.0


# ------------------------------------------------------------------------------------------------------------ cases
def listed():
    return [
        # one decode step of 16 sequences: each layer appends one K and one V row per sequence (latency)
        dict(name="token_write_step", op="token_write", B=16, N=1, Tmax=32768, d=128, ragged=False),
        # a whole 128k prompt quantised once its full layer is done
        dict(name="token_write_128k", op="token_write", B=1, N=131072, Tmax=131328, d=128, ragged=False),
        # a padded batch of prompts read back to bf16, for a later chunk's attention over them
        dict(name="token_read_32k", op="token_read", B=4, N=32768, Tmax=33000, d=64, ragged=True),
        # one decode step of 64 sequences with 8 KV heads, most pages partly filled
        dict(name="paged_write_step", op="paged_write", B=64, N=1, T=2000, Hkv=8, d=128, page=64, ragged=True),
        # ragged prompts written into the pages, starting inside a page
        dict(name="paged_write_32k", op="paged_write", B=4, N=32768, T=33001, Hkv=8, d=128, page=64, ragged=True),
        # the cached context of two sequences read back for the next chunk of their prompts
        dict(name="paged_read_64k", op="paged_read", B=2, N=65536, T=65600, Hkv=4, d=128, page=128, ragged=True),
        # a short chat turn alone on the GPU (latency)
        dict(name="paged_decode_1k", op="paged_decode", B=1, T=1000, Hq=16, Hkv=1, d=128, page=64, window=0, n_sink=0,
             ragged=False),
        # the long-context decode workload: 16 sequences of 256k tokens, 16 heads on one KV head
        dict(name="paged_decode_256k", op="paged_decode", B=16, T=262144, Hq=16, Hkv=1, d=128, page=64, window=0,
             n_sink=0, ragged=False),
        # a serving batch with grouped heads, ragged lengths, a window and sinks
        dict(name="paged_decode_gqa", op="paged_decode", B=48, T=20000, Hq=32, Hkv=8, d=64, page=32, window=4096,
             n_sink=4, ragged=True),
        # the tiny prefill's shape, window and sinks (latency)
        dict(name="window_1k", op="window_attn", B=1, Lq=1024, Lk=1024, Hq=4, Hkv=1, d=64, window=32, n_sink=4),
        # the local window of the 128k prompt: bound by reading q and writing o
        dict(name="window_128k", op="window_attn", B=1, Lq=131072, Lk=131072, Hq=16, Hkv=1, d=128, window=128, n_sink=4),
        # a later chunk of two prompts with grouped heads and a wide window: bound by the matrix products
        dict(name="window_chunk_gqa", op="window_attn", B=2, Lq=16000, Lk=40000, Hq=32, Hkv=8, d=128, window=4096,
             n_sink=16),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["token_write", "token_read", "paged_write", "paged_read", "paged_decode", "paged_decode",
                     "window_attn", "window_attn"])
    d = rng.choice([64, 128])
    if op in ("token_write", "token_read"):
        N = _log(rng, 1, 131072)
        B = _log(rng, 1, min(64, max(1, 262144 // N)))
        return dict(op=op, B=B, N=N, Tmax=N + _log(rng, 1, 5000), d=d, ragged=rng.random() < 0.5)
    page = rng.choice([16, 32, 64, 128])
    Hkv = rng.choice([1, 1, 2, 4, 8])
    if op in ("paged_write", "paged_read"):
        N = _log(rng, 1, 65536)
        B = _log(rng, 1, min(64, max(1, 131072 // (N * Hkv))))
        return dict(op=op, B=B, N=N, T=N + _log(rng, 1, 5000), Hkv=Hkv, d=d, page=page, ragged=rng.random() < 0.7)
    G = rng.choice([1, 2, 3, 4, 5, 7, 8, 16, 16])
    if op == "paged_decode":
        T = _log(rng, 1, 300000)
        B = _log(rng, 1, min(64, max(1, 2000000 // (T * Hkv))))
        window, n_sink = (0, 0) if rng.random() < 0.5 else (_log(rng, 1, 8192), rng.choice([0, 1, 4, 100]))
        return dict(op=op, B=B, T=T, Hq=G * Hkv, Hkv=Hkv, d=d, page=page, window=window, n_sink=n_sink,
                    ragged=rng.random() < 0.6)
    Lq = _log(rng, 1, 100000)
    window = _log(rng, 1, 4096)
    while Lq * G * Hkv * (window + _block(window)) > 3 * 10**9:
        Lq, window = max(1, Lq * 2 // 3), max(1, window * 3 // 4)
    B = 2 if rng.random() < 0.3 and Lq * G * Hkv * (window + _block(window)) < 10**9 else 1
    return dict(op=op, B=B, Lq=Lq, Lk=Lq + (0 if rng.random() < 0.5 else _log(rng, 1, 20000)), Hq=G * Hkv, Hkv=Hkv,
                d=d, window=window, n_sink=rng.choice([0, 0, 1, 4, 130]))


# ----------------------------------------------------------------------------------------------------------- inputs
def _gen(case, seed):
    return torch.Generator(device="cuda").manual_seed(1000003 * int(seed) + 17)


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)


def _ints(g, lo, hi, n):
    """n whole numbers in [lo, hi], int32."""
    return torch.randint(lo, hi + 1, (n,), generator=g, device="cuda", dtype=torch.int32)


def _rows(g, *shape):
    """K or V rows: normal, each token with its own size (2^-3 to 2^3), as a layer's activations have."""
    size = torch.exp2(torch.rand(*shape[:-1], 1, generator=g, device="cuda") * 6 - 3)
    return (_randn(g, *shape) * size).to(torch.bfloat16)


def _codes(g, *shape):
    """e4m3 codes of a cache that has been in use: normal values over their page's scale."""
    return (_randn(g, *shape) * 100).clamp_(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)


def _pages(g, case):
    """A pool of pages in use, and each sequence's table over it in no order."""
    B, Hkv, d, page = case["B"], case["Hkv"], case["d"], case["page"]
    mp = -(-case["T"] // page)
    P = B * mp + 3
    sc = lambda: torch.exp2(_ints(g, -9, -5, P * Hkv).float()).view(P, Hkv)  # noqa: E731
    return dict(k_pages=_codes(g, P, Hkv, page, d), v_pages=_codes(g, P, Hkv, page, d), k_scale=sc(), v_scale=sc(),
                table=torch.randperm(P, generator=g, device="cuda")[: B * mp].to(torch.int32).view(B, mp).contiguous())


def prepare(case, seed):
    g = _gen(case, seed)
    s = dict(case)
    op = case["op"]
    if op in ("token_write", "token_read", "paged_write", "paged_read"):
        B, N, d = case["B"], case["N"], case["d"]
        room = (case["Tmax"] if op[:5] == "token" else case["T"]) - N
        s["start"] = _ints(g, 0, room, B)
        s["count"] = _ints(g, min(N, max(1, N // 2)), N, B) if case["ragged"] else None
        head = () if op[:5] == "token" else (case["Hkv"],)
        if op[-5:] == "write":
            s["k"], s["v"] = _rows(g, B, N, *head, d), _rows(g, B, N, *head, d)
        else:
            s["k"], s["v"] = (torch.zeros(B, N, *head, d, dtype=torch.bfloat16, device="cuda") for _ in "kv")
    if op[:5] == "token":
        T = case["Tmax"]
        s["k_cache"], s["v_cache"] = _codes(g, B, T, d), _codes(g, B, T, d)
        s["k_scale"], s["v_scale"] = ((torch.rand(B, T, generator=g, device="cuda") + 0.5) / 100 for _ in "kv")
    elif op[:5] == "paged":
        s.update(_pages(g, case))
    if op == "paged_decode":
        B, T, Hq, Hkv, d = (case[x] for x in ("B", "T", "Hq", "Hkv", "d"))
        s["lengths"] = _ints(g, max(1, T // 4), T, B) if case["ragged"] else torch.full((B,), T, dtype=torch.int32,
                                                                                       device="cuda")
        s["q"] = (_randn(g, B, Hq, d) * 1.5).to(torch.bfloat16)
        s["o"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty(B, Hq, dtype=torch.float32, device="cuda")
    elif op == "window_attn":
        B, Lq, Lk, Hq, Hkv, d = (case[x] for x in ("B", "Lq", "Lk", "Hq", "Hkv", "d"))
        s["q"] = (_randn(g, B, Lq, Hq, d) * 1.5).to(torch.bfloat16)
        s["k"], s["v"] = _randn(g, B, Lk, Hkv, d).to(torch.bfloat16), _randn(g, B, Lk, Hkv, d).to(torch.bfloat16)
        s["o"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty(B, Lq, Hq, dtype=torch.float32, device="cuda")
    return s


# ------------------------------------------------------------------------------------------------------ plain forms
def _places(s):
    """[B, N] cache positions of the rows, and which of them are there."""
    N = s["k"].shape[1]
    i = torch.arange(N, device="cuda")
    there = i < (s["count"] if s["count"] is not None else torch.full_like(s["start"], N)).unsqueeze(1)
    return s["start"].long().unsqueeze(1) + i, there


def _token_write(s):
    pos, there = _places(s)
    b = torch.arange(s["B"], device="cuda").unsqueeze(1).expand_as(pos)
    b, pos = b[there], pos[there]
    for x, cache, scale in ((s["k"], s["k_cache"], s["k_scale"]), (s["v"], s["v_cache"], s["v_scale"])):
        x = x[there].float()
        top = x.abs().amax(-1)
        sc = torch.where(top > 0, top / E4M3_MAX, torch.ones_like(top))
        cache.view(torch.uint8)[b, pos] = (x / sc.unsqueeze(-1)).clamp(-E4M3_MAX, E4M3_MAX).to(
            torch.float8_e4m3fn).view(torch.uint8)
        scale[b, pos] = sc
    return s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"]


def _token_read(s):
    pos, there = _places(s)
    b = torch.arange(s["B"], device="cuda").unsqueeze(1)
    pos = pos.clamp(max=s["Tmax"] - 1)
    for x, cache, scale in ((s["k"], s["k_cache"], s["k_scale"]), (s["v"], s["v_cache"], s["v_scale"])):
        rows = cache.view(torch.uint8)[b, pos].view(torch.float8_e4m3fn).float() * scale[b, pos].unsqueeze(-1)
        x.copy_(torch.where(there.unsqueeze(-1), rows.to(torch.bfloat16), x))
    return s["k"], s["v"]


def _power(top):
    """The least power of two p >= 2^-126 with top <= 448 p."""
    m, e = torch.frexp(top)
    e = torch.where(m > 0.875, e - 8, e - 9)
    return torch.ldexp(torch.ones_like(top), torch.where(top > 0, e, torch.full_like(e, -126)).clamp(min=-126))


def _paged_write(s):
    B, N, page, Hkv, d = s["B"], s["N"], s["page"], s["Hkv"], s["d"]
    start = s["start"].long().view(B, 1, 1)
    end = start + (s["count"].long().view(B, 1, 1) if s["count"] is not None else N)
    J = (N + page - 2) // page + 1                                  # pages that N rows can touch
    slot = start[:, :, 0] // page + torch.arange(J, device="cuda")  # [B, J]
    t = slot.unsqueeze(-1) * page + torch.arange(page, device="cuda")  # [B, J, page]
    new, old = (t >= start) & (t < end), t < start
    touched = new.any(-1)
    pid = torch.gather(s["table"], 1, slot.clamp(max=s["table"].shape[1] - 1)).long()  # [B, J]
    b = torch.arange(B, device="cuda").view(B, 1, 1)
    for x, pages, scale in ((s["k"], s["k_pages"], s["k_scale"]), (s["v"], s["v_pages"], s["v_scale"])):
        x = x[b, (t - start).clamp(0, N - 1)].permute(0, 1, 3, 2, 4).float()        # [B, J, Hkv, page, d]
        is_new, is_old = new[:, :, None, :, None], old[:, :, None, :, None]
        was = pages.view(torch.uint8)[pid].view(torch.float8_e4m3fn)
        had = scale[pid]                                                            # [B, J, Hkv]
        sc = _power(torch.where(is_new, x.abs(), torch.zeros_like(x)).amax((-1, -2)))
        sc = torch.where(old.any(-1, keepdim=True), torch.maximum(sc, had), sc)
        val = torch.where(is_new, x, was.float() * had[..., None, None]) / sc[..., None, None]
        code = val.clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).view(torch.uint8)
        code = torch.where(is_new | is_old, code, was.view(torch.uint8))
        pages.view(torch.uint8)[pid[touched]] = code[touched]
        scale[pid[touched]] = sc[touched]
    return s["k_pages"], s["v_pages"], s["k_scale"], s["v_scale"]


def _paged_read(s):
    pos, there = _places(s)
    page = s["page"]
    pos = pos.clamp(max=s["table"].shape[1] * page - 1)
    pid = torch.gather(s["table"], 1, pos // page).long()
    for x, pages, scale in ((s["k"], s["k_pages"], s["k_scale"]), (s["v"], s["v_pages"], s["v_scale"])):
        rows = pages.view(torch.uint8)[pid, :, pos % page].view(torch.float8_e4m3fn).float() * scale[pid].unsqueeze(-1)
        x.copy_(torch.where(there[..., None, None], rows.to(torch.bfloat16), x))
    return s["k"], s["v"]


def _paged_decode(s):
    B, Hq, Hkv, d = s["B"], s["Hq"], s["Hkv"], s["d"]
    G = Hq // Hkv
    table = s["table"].long()

    def cache(pages, scale):  # [B, Hkv, T, d]
        x = pages.view(torch.uint8)[table].view(torch.float8_e4m3fn).float() * scale[table][..., None, None]
        return x.permute(0, 2, 1, 3, 4).reshape(B, Hkv, -1, d)

    q = s["q"].float().view(B, Hkv, G, d)
    x = torch.matmul(q, cache(s["k_pages"], s["k_scale"]).transpose(-1, -2)) / math.sqrt(d)
    pos = torch.arange(x.shape[-1], device="cuda")
    T = s["lengths"].view(B, 1)
    seen = pos < T
    if s["window"]:
        seen = seen & ((pos >= T - s["window"]) | (pos < s["n_sink"]))
    x = torch.where(seen.view(B, 1, 1, -1), x, torch.full_like(x, -math.inf))
    m = x.amax(-1, keepdim=True)
    p = torch.exp(x - m)
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p, cache(s["v_pages"], s["v_scale"])) / total
    return o.view(B, Hq, d).to(torch.bfloat16), (m + torch.log(total)).view(B, Hq)


def _block(window):
    """Query rows taken together by the plain window."""
    return max(64, min(512, window))


def _window_attn(s):
    q, k, v = s["q"], s["k"], s["v"]
    B, Lq, Hq, d = q.shape
    Lk, Hkv = k.shape[1], k.shape[2]
    G, C, W = Hq // Hkv, _block(s["window"]), min(s["window"], Lk)
    C = min(C, Lq)
    nb = -(-Lq // C)
    i = torch.arange(nb, device="cuda").unsqueeze(1) * C
    t = Lk - Lq + i + torch.arange(C, device="cuda")                         # [nb, C] positions of the queries
    near = Lk - Lq + i - (W - 1) + torch.arange(C + W - 1, device="cuda")    # [nb, C + W - 1] keys of a block
    first = torch.arange(min(s["n_sink"], Lk), device="cuda")
    qb = q.float()[:, (i + torch.arange(C, device="cuda")).clamp(max=Lq - 1)]      # [B, nb, C, Hq, d]
    qb = qb.view(B, nb, C, Hkv, G, d).permute(0, 1, 3, 2, 4, 5).reshape(B, nb, Hkv, C * G, d)
    at = near.clamp(0, Lk - 1)
    kb, vb = (z[:, at].float().permute(0, 1, 3, 2, 4) for z in (k, v))             # [B, nb, Hkv, M, d]
    ks, vs = (z[:, first].float().permute(0, 2, 1, 3).unsqueeze(1) for z in (k, v))  # [B, 1, Hkv, ns, d]
    tt, nn = t.unsqueeze(-1), near.unsqueeze(1)
    see = (nn >= 0) & (nn <= tt) & (nn > tt - s["window"])
    see_first = first <= tt - s["window"]                                          # those in the window count there
    spread = lambda z: z.unsqueeze(2).expand(nb, C, G, -1).reshape(nb, 1, C * G, -1)  # noqa: E731
    x = torch.matmul(qb, kb.transpose(-1, -2)).div_(math.sqrt(d)).masked_fill_(~spread(see), -math.inf)
    y = torch.matmul(qb, ks.transpose(-1, -2)).div_(math.sqrt(d)).masked_fill_(~spread(see_first), -math.inf)
    m = x.amax(-1, keepdim=True)
    m = torch.maximum(m, y.amax(-1, keepdim=True)) if len(first) else m
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)                        # rows past the last query
    x.sub_(m).exp_()
    y.sub_(m).exp_()
    total = x.sum(-1, keepdim=True) + y.sum(-1, keepdim=True)
    o = (torch.matmul(x, vb) + torch.matmul(y, vs)) / total

    def back(z):  # [B, nb, Hkv, C * G, n] -> [B, Lq, Hq, n]
        z = z.view(B, nb, Hkv, C, G, -1).permute(0, 1, 3, 2, 4, 5)
        return z.reshape(B, nb * C, Hq, -1)[:, :Lq].contiguous()

    return back(o).to(torch.bfloat16), back(m + torch.log(total)).squeeze(-1)


def _own(s):
    import token_level_top_hs2_b200 as hs2
    op = s["op"]
    if op == "token_write":
        hs2.hs2_kv_write(s["k"], s["v"], s["start"], s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"],
                         count=s["count"])
        return s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"]
    if op == "token_read":
        return hs2.hs2_kv_read(s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"], s["start"], s["N"],
                               count=s["count"], k=s["k"], v=s["v"])
    if op == "paged_write":
        hs2.hs2_paged_kv_write(s["k"], s["v"], s["table"], s["start"], s["k_pages"], s["v_pages"], s["k_scale"],
                               s["v_scale"], count=s["count"])
        return s["k_pages"], s["v_pages"], s["k_scale"], s["v_scale"]
    if op == "paged_read":
        return hs2.hs2_paged_kv_read(s["k_pages"], s["v_pages"], s["k_scale"], s["v_scale"], s["table"], s["start"],
                                     s["N"], count=s["count"], k=s["k"], v=s["v"])
    if op == "paged_decode":
        return hs2.hs2_paged_decode(s["q"], s["k_pages"], s["v_pages"], s["k_scale"], s["v_scale"], s["table"],
                                    s["lengths"], window=s["window"] or None, n_sink=s["n_sink"], o=s["o"],
                                    lse=s["lse"])
    return hs2.hs2_window_attn(s["q"], s["k"], s["v"], s["window"], s["n_sink"], o=s["o"], lse=s["lse"])


def run(state):
    if own:
        return _own(state)
    return {"token_write": _token_write, "token_read": _token_read, "paged_write": _paged_write,
            "paged_read": _paged_read, "paged_decode": _paged_decode, "window_attn": _window_attn}[state["op"]](state)


# ------------------------------------------------------------------------------------------------------------- work
def _seen(t, window, n_sink):
    """Keys that a query at position t sees."""
    return min(t + 1, window) + max(0, min(n_sink, t + 1 - window))


def work(case):
    op = case["op"]
    if op in ("token_write", "token_read", "paged_write", "paged_read"):
        heads = case.get("Hkv", 1)
        n = case["B"] * case["N"] * (0.75 if case["ragged"] and case["N"] > 1 else 1)  # rows there, on average
        scales = n if op[:5] == "token" else n / case["page"]
        return {"bytes": n * heads * 2 * case["d"] * 3 + 2 * scales * heads * 4, "flops": 0}
    Hq, Hkv, d = case["Hq"], case["Hkv"], case["d"]
    if op == "paged_decode":
        T = case["T"] * (0.625 if case["ragged"] else 1)
        n = case["B"] * (min(T, case["window"] + case["n_sink"]) if case["window"] else T)
        return {"bytes": n * Hkv * 2 * (d + 4 / case["page"]) + case["B"] * Hq * d * 4, "flops": 4 * n * Hq * d}
    B, Lq, Lk, W, ns = (case[x] for x in ("B", "Lq", "Lk", "window", "n_sink"))
    lo = Lk - Lq
    pairs = sum(_seen(t, W, ns) for t in range(lo, min(Lk, max(lo, W + ns))))
    pairs += max(0, Lk - max(lo, W + ns)) * _seen(Lk, W, ns)
    keys = min(Lk, Lq + W + ns)
    return {"bytes": B * (Lq * Hq * (4 * d + 4) + keys * Hkv * 4 * d), "flops": 4 * B * pairs * Hq * d}


# ------------------------------------------------------------------------------------------------ values in 64 bits
def _e4m3(x):
    """Nearest e4m3 value, ties to even, saturated: steps of 2^(e-3) for 2^e <= |x| < 2^(e+1), 2^-9 below 2^-6."""
    e = torch.frexp(x.abs().clamp(min=2.0**-6))[1].double() - 1
    step = torch.exp2(e - 3)
    return (torch.round(x / step) * step).clamp(-E4M3_MAX, E4M3_MAX)


def _exact_write(s):
    token = s["op"] == "token_write"
    names = ("k_cache", "v_cache") if token else ("k_pages", "v_pages")
    out, scales = [s[n].float().double() for n in names], [s["k_scale"].double(), s["v_scale"].double()]
    counts = s["count"].tolist() if s["count"] is not None else [s["N"]] * s["B"]
    for b, (lo, n) in enumerate(zip(s["start"].tolist(), counts)):
        for x, cache, sc in zip((s["k"], s["v"]), out, scales):
            x = x[b, :n].double()
            if token:
                top = x.abs().amax(-1)
                sc[b, lo:lo + n] = torch.where(top > 0, top / E4M3_MAX, 1.0)
                cache[b, lo:lo + n] = _e4m3(x / sc[b, lo:lo + n, None])
                continue
            page, table = s["page"], s["table"][b].tolist()
            inner = range(-(-lo // page), (lo + n) // page)  # pages that the rows fill
            rest = [j for j in range(lo // page, -(-(lo + n) // page)) if j not in inner]
            for j in rest:
                t0, t1 = max(lo, j * page), min(lo + n, (j + 1) * page)
                pid, at = table[j], t0 - j * page
                new = x[t0 - lo:t1 - lo].transpose(0, 1)  # [Hkv, n, d]
                had = sc[pid].clone()
                size = new.abs().amax((-1, -2))
                p = torch.exp2(torch.ceil(torch.log2(size / E4M3_MAX)).clamp(min=-126))
                p = torch.maximum(p, had) if at else p
                if at:
                    cache[pid, :, :at] = _e4m3(cache[pid, :, :at] * (had / p)[:, None, None])
                cache[pid, :, at:at + t1 - t0] = _e4m3(new / p[:, None, None])
                sc[pid] = p
            if len(inner):
                pid = s["table"][b, inner.start:inner.stop].long()
                new = x[inner.start * page - lo:inner.stop * page - lo]
                new = new.view(len(inner), page, s["Hkv"], -1).transpose(1, 2)
                p = torch.exp2(torch.ceil(torch.log2(new.abs().amax((-1, -2)) / E4M3_MAX)).clamp(min=-126))
                cache[pid], sc[pid] = _e4m3(new / p[..., None, None]), p
    return [*out, *scales]


def _exact_read(s):
    counts = s["count"].tolist() if s["count"] is not None else [s["N"]] * s["B"]
    out = []
    for x, kv in ((s["k"], "k"), (s["v"], "v")):
        x, sc = x.double(), s[kv + "_scale"].double()
        for b, (lo, n) in enumerate(zip(s["start"].tolist(), counts)):
            if s["op"] == "token_read":
                x[b, :n] = s[kv + "_cache"][b, lo:lo + n].float().double() * sc[b, lo:lo + n, None]
            else:
                a = lo // s["page"]
                pid = s["table"][b, a:-(-(lo + n) // s["page"])].long()
                whole = s[kv + "_pages"].view(torch.uint8)[pid].view(torch.float8_e4m3fn).float().double()
                whole = (whole * sc[pid][..., None, None]).transpose(1, 2).flatten(0, 1)
                x[b, :n] = whole[lo - a * s["page"]:][:n]
        out.append(x)
    return out


def _softmax_rows(x, v):
    """x [..., n] logits, v [..., n, d]: the weighted mean and the log of the sum."""
    lse = torch.logsumexp(x, -1)
    return torch.matmul(torch.exp(x - lse.unsqueeze(-1)), v), lse


def exact(case, seed):
    s = prepare(case, seed)
    op = s["op"]
    if op in ("token_write", "paged_write"):
        return _exact_write(s)
    if op in ("token_read", "paged_read"):
        return _exact_read(s)
    Hq, Hkv, d = s["Hq"], s["Hkv"], s["d"]
    G = Hq // Hkv
    if op == "paged_decode":
        o = torch.empty(s["B"], Hq, d, dtype=torch.float64, device="cuda")
        lse = torch.empty(s["B"], Hq, dtype=torch.float64, device="cuda")
        for b, T in enumerate(s["lengths"].tolist()):
            pos = torch.arange(T, device="cuda")
            if s["window"]:
                pos = pos[(pos >= T - s["window"]) | (pos < s["n_sink"])]
            pid = s["table"][b].long()[pos // s["page"]]
            for h in range(Hkv):
                k, v = (s[z + "_pages"].view(torch.uint8)[pid, h, pos % s["page"]].view(torch.float8_e4m3fn).float()
                        .double() * s[z + "_scale"].double()[pid, h, None] for z in "kv")
                x = s["q"][b, h * G:(h + 1) * G].double() @ k.T / math.sqrt(d)
                o[b, h * G:(h + 1) * G], lse[b, h * G:(h + 1) * G] = _softmax_rows(x, v)
        return o, lse
    B, Lq, Lk, W, ns = (case[x] for x in ("B", "Lq", "Lk", "window", "n_sink"))
    o = torch.empty(B, Lq, Hq, d, dtype=torch.float64, device="cuda")
    lse = torch.empty(B, Lq, Hq, dtype=torch.float64, device="cuda")
    step = 2048
    for r0 in range(0, Lq, step):
        r1 = min(Lq, r0 + step)
        t = torch.arange(Lk - Lq + r0, Lk - Lq + r1, device="cuda")
        lo = max(0, Lk - Lq + r0 - W + 1)
        at = torch.cat([torch.arange(min(ns, lo), device="cuda"), torch.arange(lo, Lk - Lq + r1, device="cuda")])
        hide = (at > t[:, None]) | ((at <= t[:, None] - W) & (at >= ns))
        for h in range(Hkv):
            q = s["q"][:, r0:r1, h * G:(h + 1) * G].double().permute(0, 2, 1, 3)       # [B, G, n, d]
            k, v = s["k"][:, at, h].double().unsqueeze(1), s["v"][:, at, h].double().unsqueeze(1)
            x = (q @ k.transpose(-1, -2) / math.sqrt(d)).masked_fill(hide, -math.inf)
            a, b = _softmax_rows(x, v)
            o[:, r0:r1, h * G:(h + 1) * G], lse[:, r0:r1, h * G:(h + 1) * G] = a.permute(0, 2, 1, 3), b.transpose(1, 2)
    return o, lse

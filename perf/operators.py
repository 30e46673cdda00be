"""The paged Q3 KV-cache operators: what is measured, and their plain forms.

Three operators, used one after another in a serving step:

  tables  block tables and slot maps from request lengths (hlwq_kv_block_tables)
  append  new keys and values: what leaves the exact window is encoded into
          pages, the most recent tokens stay exact (hlwq_kv_paged_append)
  attend  causal attention of the new tokens over the paged cache
          (hlwq_kv_paged_attention)

A request has `past` tokens cached and `new` tokens in this step.  Of N tokens
the last min(N, R) are kept in bfloat16 in a ring of R slots (token i in slot
i % R), the N - R before them as 3-bit codes of the rotated unit vector with a
binary16 norm, in pages of P tokens.
"""

import math
import random

import torch

own = False

D = 256      # head_dim of the encoding
NBYTES = 96  # 256 codes of 3 bits


# ------------------------------------------------------------------ cases
def listed():
    return [
        # the smallest step of a serving loop: eight decoding requests
        dict(name="tables decode 8", op="tables", B=8, past_lo=10, past_hi=2000, new_lo=1, new_hi=1, P=64, R=128, pad=0),
        # a full decode batch; the slot map is padded as for a captured graph
        dict(name="tables decode 512", op="tables", B=512, past_lo=1, past_hi=16384, new_lo=1, new_hi=1, P=16, R=128,
             pad=13),
        # prompts of many lengths arriving together
        dict(name="tables prompts 32", op="tables", B=32, past_lo=0, past_hi=0, new_lo=100, new_hi=8192, P=64, R=128,
             pad=0),
        # one token of one request
        dict(name="append one token", op="append", B=1, past_lo=1000, past_hi=1000, new_lo=1, new_hi=1, H=4, P=64, R=128),
        # a decode batch: each row moves one token out of its window
        dict(name="append decode 256", op="append", B=256, past_lo=60, past_hi=4000, new_lo=1, new_hi=1, H=4, P=16,
             R=128),
        # prompt chunks, 16 thousand tokens or so
        dict(name="append chunks 6", op="append", B=6, past_lo=0, past_hi=5000, new_lo=1000, new_hi=5000, H=4, P=64,
             R=128),
        # one short request decoding: latency
        dict(name="attend decode 1x300", op="attend", B=1, past_lo=299, past_hi=299, new_lo=1, new_hi=1, H=4, G=6, P=64,
             R=128),
        # one long context decoding: the keys have to be split over the machine
        dict(name="attend decode 1x131071", op="attend", B=1, past_lo=131070, past_hi=131070, new_lo=1, new_hi=1, H=4,
             G=6, P=64, R=128),
        # a decode batch with contexts of very different lengths
        dict(name="attend decode 64", op="attend", B=64, past_lo=64, past_hi=16383, new_lo=1, new_hi=1, H=4, G=6, P=64,
             R=128),
        # a few drafted tokens per request to verify, no exact window, small pages
        dict(name="attend draft 16", op="attend", B=16, past_lo=100, past_hi=7001, new_lo=2, new_hi=4, H=8, G=4, P=16,
             R=0),
        # one chunk of a long prompt
        dict(name="attend chunk 2048", op="attend", B=1, past_lo=6145, past_hi=6145, new_lo=2048, new_hi=2048, H=4, G=6,
             P=64, R=128),
        # chunks of many lengths, some requests at their first token and some late
        dict(name="attend chunks 8", op="attend", B=8, past_lo=0, past_hi=4000, new_lo=1, new_hi=1501, H=2, G=8, P=128,
             R=64),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["tables", "append", "attend", "attend"])
    P = rng.choice([16, 48, 64, 128, 256])
    R = rng.choice([0, 1, 31, 64, 128, 128, 128])
    if op == "tables":
        B = _log(rng, 1, 512)
        if rng.random() < 0.5:
            return dict(op=op, B=B, past_lo=0, past_hi=R + _log(rng, 10, 16384), new_lo=0, new_hi=rng.choice([1, 1, 5]), P=P,
                        R=R, pad=rng.choice([1, 7, 64]))
        hi = min(8192, _log(rng, 20, 100000 // B + 21))
        return dict(op=op, B=B, past_lo=0, past_hi=R + _log(rng, 10, 4000), new_lo=1, new_hi=hi, P=P, R=R,
                    pad=rng.choice([0, 1, 100]))
    H = rng.choice([1, 2, 4, 5, 8])
    if op == "append":
        B = _log(rng, 1, 256)
        hi = max(1, min(5000, _log(rng, 1, 40000 // (B * H) + 2)))
        return dict(op=op, B=B, past_lo=0, past_hi=_log(rng, 10, min(5000, 1000000 // (B * H))), new_lo=min(1, hi),
                    new_hi=hi, H=H, P=P, R=R)
    G = rng.choice([1, 2, 3, 4, 6, 8, 16])
    if rng.random() < 0.5:
        # decoding, or verifying a few drafted tokens
        B = _log(rng, 1, 64)
        hi = max(200, min(100000, _log(rng, 200, 1500000 // (B * H))))
        return dict(op=op, B=B, past_lo=rng.choice([0, hi // 3, hi]), past_hi=hi, new_lo=1, new_hi=rng.choice([1, 1, 1, 3]),
                    H=H, G=G, P=P, R=R)
    B = rng.choice([1, 1, 2, 5])
    hi = _log(rng, 17, 6000 // B)
    # the padded plain form holds B * H * G * new * keys scores
    ctx = max(10, min(8000, int(3e8 / (B * H * G * hi)) - hi))
    return dict(op=op, B=B, past_lo=0, past_hi=_log(rng, 10, max(11, ctx)), new_lo=rng.choice([1, hi]), new_hi=hi, H=H, G=G,
                P=P, R=R)


def _lens(case):
    """The requests' (past, new): spread over the case's ranges, the same for every seed; the first request has the
    largest of both, the last the smallest."""
    rng = random.Random("%(B)d %(past_lo)d %(past_hi)d %(new_lo)d %(new_hi)d" % case)
    B = case["B"]
    past = [rng.randint(case["past_lo"], case["past_hi"]) for _ in range(B)]
    new = [rng.randint(case["new_lo"], case["new_hi"]) for _ in range(B)]
    past[0], new[0] = case["past_hi"], case["new_hi"]
    if B > 1:
        past[-1], new[-1] = case["past_lo"], case["new_lo"]
    return past, new


def _enc(n, R):
    return max(0, n - R)


def _pages(n, P, R):
    return -(-_enc(n, R) // P)


def work(case):
    past, new = _lens(case)
    R, P, op = case["R"], case["P"], case["op"]
    T = sum(new)
    if op == "tables":
        got = sum(_pages(p + n, P, R) - _pages(p, P, R) for p, n in zip(past, new))
        # a request's slots lie in these pages: their table entries are read unless they are new
        used = sum(_pages(p + n, P, R) - _enc(p, R) // P for p, n in zip(past, new))
        return {"bytes": 8 * len(past) + 4 * (len(past) + 1) + 8 * (T + case["pad"]) + 8 * got + 4 * max(0, used - got) + 8,
                "flops": 0}
    H = case["H"]
    if op == "append":
        leave = sum(_enc(p + n, R) - _enc(p, R) for p, n in zip(past, new))
        old = sum(min(_enc(p + n, R), p) - _enc(p, R) for p, n in zip(past, new))  # those that leave from the ring
        stay = sum(min(n, R) for n in new)
        return {"bytes": 2 * H * (512 * T + 512 * old + 98 * leave + 512 * stay) + 8 * T + 4 * (2 * len(past) + 1),
                "flops": 2 * H * leave * (256 * 8 + 512 + 256)}
    Hq, kv, fl = H * case["G"], 0, 0
    for p, n in zip(past, new):
        e = _enc(p + n, R)
        kv += 196 * e + 1024 * (p + n - e) + (4 * -(-e // P)) // H
        fl += n * p + n * (n + 1) // 2
    return {"bytes": H * kv + 2 * 512 * Hq * T + 4 * (2 * len(past) + 1), "flops": 4 * 256 * Hq * fl}


# ------------------------------------------------------------------ what a program has in hand
def _centroids(dtype):
    """The 8-level Lloyd-Max quantizer of N(0, 1) as binary32 values, from its fixed point."""
    c = [0.25, 0.75, 1.4, 2.2]
    pdf = lambda x: math.exp(-x * x / 2) / math.sqrt(2 * math.pi)  # noqa: E731
    cdf = lambda x: 0.5 * math.erfc(-x / math.sqrt(2))  # noqa: E731
    for _ in range(2000):
        b = [0.0] + [(c[k] + c[k + 1]) / 2 for k in range(3)] + [math.inf]
        c = [(pdf(b[k]) - pdf(b[k + 1])) / (cdf(b[k + 1]) - cdf(b[k])) for k in range(4)]
    half = torch.tensor(c, dtype=torch.float64).to(torch.float32)
    return torch.cat([-half.flip(0), half]).to(dtype).cuda()


def _hadamard(dtype):
    h = torch.ones(1, 1, dtype=dtype, device="cuda")
    while h.shape[0] < D:
        h = torch.cat([torch.cat([h, h], 1), torch.cat([h, -h], 1)], 0)
    return h


def _pack(codes):
    """codes [..., 256] of 0..7 -> bytes [..., 96], three bits each, lowest first."""
    c = codes.to(torch.int32).reshape(*codes.shape[:-1], D // 8, 8)
    w = (c << torch.arange(0, 24, 3, dtype=torch.int32, device=c.device)).sum(-1, dtype=torch.int32)
    return torch.stack([w & 255, (w >> 8) & 255, w >> 16], -1).to(torch.uint8).reshape(*codes.shape[:-1], NBYTES)


def _codes(packed):
    """bytes [..., 96] -> codes [..., 256] (int32)."""
    b = packed.to(torch.int32).reshape(*packed.shape[:-1], D // 8, 3)
    w = b[..., 0] | (b[..., 1] << 8) | (b[..., 2] << 16)
    c = (w.unsqueeze(-1) >> torch.arange(0, 24, 3, dtype=torch.int32, device=w.device)) & 7
    return c.reshape(*packed.shape[:-1], D)


def _cached(g, shape, spread):
    """Encoded vectors as a cache holds them: the rotated coordinates of a key or value are near N(0, 1), its length varies
    (lognormal) around 16."""
    n = math.prod(shape)
    c = _centroids(torch.float32)
    mid = (c[1:] + c[:-1]) / 2
    packed = torch.empty(n, NBYTES, dtype=torch.uint8, device="cuda")
    norms = torch.empty(n, dtype=torch.float16, device="cuda")
    for i in range(0, n, 1 << 18):
        m = min(1 << 18, n - i)
        z = torch.randn(m, D, generator=g, device="cuda")
        packed[i:i + m] = _pack(torch.bucketize(z, mid, out_int32=True))
        norms[i:i + m] = 16 * torch.exp(spread * torch.randn(m, generator=g, device="cuda"))
    return packed.reshape(*shape, NBYTES), norms.view(torch.uint16).reshape(shape)


def _ints(v, dtype=torch.int32):
    return torch.tensor(v, dtype=dtype, device="cuda")


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    past, new = _lens(case)
    op, B, P, R = case["op"], case["B"], case["P"], case["R"]
    T = sum(new)
    s = dict(op=op, P=P, R=R, past=past, new=new, n_past=_ints(past), n_new=_ints(new), max_new=max(new))
    need = sum(_pages(p + n, P, R) for p, n in zip(past, new))
    held = sum(_pages(p, P, R) for p in past)
    width = max(1, max(_pages(p + n, P, R) for p, n in zip(past, new)) + 3)
    s["num_pages"] = need + (500 if op == "tables" else 5)
    order = torch.randperm(s["num_pages"], generator=g, device="cuda").to(torch.int32)  # pages in the order of their use
    # the pool as after some time of serving: pages of all requests interleaved
    tab = torch.full((B, width), -1, dtype=torch.int32)
    at, lo = 0, order.cpu()
    for b, (p, n) in enumerate(zip(past, new)):
        k = _pages(p if op == "tables" else p + n, P, R)
        tab[b, :k] = lo[at:at + k]
        at += k
    s["table"] = tab.cuda()
    if op == "tables":
        s["free"] = order[held:].contiguous()
        s["n_free"] = _ints([s["num_pages"] - held])
        s["T"] = T + case["pad"]
        s.update(n_free_out=_ints([0]), cu=torch.zeros(B + 1, dtype=torch.int32, device="cuda"),
                 slots=torch.zeros(s["T"], dtype=torch.int64, device="cuda"))
        return s
    H = case["H"]
    s["H"] = H
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    s["cu"] = _ints(cu)
    s["cb8"], s["had"] = _centroids(torch.float32), _hadamard(torch.float64)
    bf = lambda *shape: torch.randn(*shape, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
    if R:
        s["kwin"], s["vwin"] = bf(B, H, R, D), bf(B, H, R, D)
    else:
        s["kwin"] = s["vwin"] = None
    if op == "append":
        s["K"], s["V"] = bf(T, H, D), bf(T, H, D)
        s["K"][..., :3] *= 20  # keys have a few large channels
        b = torch.repeat_interleave(torch.arange(B, device="cuda"), s["n_new"].long(), output_size=T)
        i = s["n_past"].long()[b] + torch.arange(T, device="cuda") - s["cu"].long()[b] - R
        page = s["table"][b, torch.div(i.clamp(min=0), P, rounding_mode="floor")].long()
        s["slots"] = torch.where(i >= 0, page * P + i.clamp(min=0) % P, -1)
        shape = (s["num_pages"], H, P)
        for x in "kv":
            s[x + "p"] = torch.zeros(*shape, NBYTES, dtype=torch.uint8, device="cuda")
            s[x + "n"] = torch.zeros(shape, dtype=torch.uint16, device="cuda")
        return s
    s["G"] = case["G"]
    s["kp"], s["kn"] = _cached(g, (s["num_pages"], H, P), 0.3)
    s["vp"], s["vn"] = _cached(g, (s["num_pages"], H, P), 0.3)
    s["Q"] = bf(T, H * case["G"], D)
    s["Q"] *= 1.5
    s["out"] = torch.empty_like(s["Q"])
    return s


# ------------------------------------------------------------------ one pass
def run(state):
    s = state
    if own:
        from dequant_matmul_b200 import hlwq
        if s["op"] == "tables":
            hlwq.kv_block_tables(s["n_past"], s["n_new"], s["free"], s["n_free"], s["table"], s["P"], s["R"],
                                 n_free_out=s["n_free_out"], cu_new=s["cu"], slot_map=s["slots"])
            return dict(table=s["table"], cu=s["cu"], slots=s["slots"], n_free=s["n_free_out"])
        win = (s["kwin"], s["vwin"]) if s["R"] else None
        if s["op"] == "append":
            hlwq.kv_paged_append(s["K"], s["V"], s["slots"], s["cu"], s["n_past"], (s["kp"], s["kn"]), (s["vp"], s["vn"]),
                                 win, s["cb8"])
            return _cache_out(s)
        if "ws" not in s:
            s["ws"] = torch.empty(hlwq.kv_attention_workspace(s["Q"], s["H"], len(s["past"]), s["max_new"]),
                                  dtype=torch.uint8, device="cuda")
        return hlwq.kv_paged_attention(s["Q"], s["cu"], s["n_past"], s["table"], (s["kp"], s["kn"]), (s["vp"], s["vn"]), win,
                                       s["cb8"], s["max_new"], out=s["out"], workspace=s["ws"])
    return {"tables": _plain_tables, "append": _plain_append, "attend": _plain_attend}[s["op"]](s)


def _cache_out(s):
    # the packed bytes are whole numbers, held to be equal; the norms are binary16 values
    r = dict(kp=s["kp"], kn=s["kn"].view(torch.float16), vp=s["vp"], vn=s["vn"].view(torch.float16))
    if s["R"]:
        r.update(kwin=s["kwin"], vwin=s["vwin"])
    return r


def _up(n, P, R):
    """Pages of the encoded tokens of n tokens."""
    return torch.div((n - R).clamp(min=0) + P - 1, P, rounding_mode="floor")


def _token_rows(cu, T):
    """The request of each of T tokens (the last one's for tokens behind them), and its place among the request's."""
    t = torch.arange(T, device="cuda")
    b = torch.searchsorted(cu[1:].long(), t, right=True).clamp(max=cu.numel() - 2)
    return b, t - cu.long()[b]


def _plain_tables(s):
    P, R = s["P"], s["R"]
    past, new = s["n_past"].long(), s["n_new"].long()
    s["cu"][1:] = new.cumsum(0)
    old, want = _up(past, P, R), _up(past + new, P, R)
    need = want - old
    first = need.cumsum(0) - need
    j = torch.arange(s["table"].shape[1], device="cuda")
    fresh = (j >= old[:, None]) & (j < want[:, None])
    k = s["n_free"].long() - 1 - (first[:, None] + j - old[:, None])
    s["table"].copy_(torch.where(fresh, s["free"][k.clamp(0, s["free"].numel() - 1)], s["table"]))
    s["n_free_out"].copy_(s["n_free"] - need.sum())
    b, at = _token_rows(s["cu"], s["T"])
    i = past[b] + at - R
    page = s["table"][b, torch.div(i, P, rounding_mode="floor").clamp(0, s["table"].shape[1] - 1)].long()
    live = (i >= 0) & (torch.arange(s["T"], device="cuda") < s["cu"][-1])
    s["slots"].copy_(torch.where(live, page * P + i % P, -1))
    return dict(table=s["table"], cu=s["cu"], slots=s["slots"], n_free=s["n_free_out"])


def _half(n):
    """binary64 -> the nearest binary16, ties to even, without a rounding to binary32 between."""
    unit = torch.exp2((torch.frexp(n).exponent - 11).clamp(min=-24).double())
    return (torch.round(n / unit) * unit).to(torch.float16)


def _encode(x, cb8, had):
    """x [N, 256] -> (packed, norms): in 64 bits, since codes depend on which side of a border a value lies."""
    x = x.double()
    n = (x * x).sum(-1).sqrt()
    y = x @ had / torch.where(n > 0, n, 1.0)[:, None]
    c = cb8.double()
    codes = torch.bucketize(y, (c[1:] + c[:-1]) / 2, out_int32=True)  # how many borders lie below y
    return _pack(codes), _half(n)


def _plain_append(s):
    P, R, H = s["P"], s["R"], s["H"]
    T = s["K"].shape[0]
    b, j = _token_rows(s["cu"], T)
    past, new = s["n_past"].long()[b], (s["cu"][1:] - s["cu"][:-1]).long()[b]
    goes = s["slots"] >= 0
    slot = s["slots"][goes]
    page, at = torch.div(slot, P, rounding_mode="floor"), slot % P
    for x, packed, norms, win in ((s["K"], s["kp"], s["kn"], s["kwin"]), (s["V"], s["vp"], s["vn"], s["vwin"])):
        src = x
        if R:
            here = (j >= R)[:, None, None]
            before = win[b, :, ((past + j) % R)]  # token past + j - R is in the slot of token past + j
            src = torch.where(here, x[(torch.arange(T, device="cuda") - R).clamp(min=0)], before)
        p, n = _encode(src[goes].reshape(-1, D), s["cb8"], s["had"])
        packed[page, :, at] = p.reshape(-1, H, NBYTES)
        norms.view(torch.float16)[page, :, at] = n.reshape(-1, H)
        if R:
            stays = j >= new - R
            win[b[stays], :, ((past + j) % R)[stays]] = x[stays]
    return _cache_out(s)


def _plain_attend(s):
    P, R, H, G = s["P"], s["R"], s["H"], s["G"]
    Q, T, B = s["Q"], s["Q"].shape[0], s["n_past"].numel()
    past, new = s["n_past"].long(), (s["cu"][1:] - s["cu"][:-1]).long()
    total = past + new
    enc = (total - R).clamp(min=0)
    L = max(p + n for p, n in zip(s["past"], s["new"]))
    i = torch.arange(L, device="cuda")
    page = s["table"][:, torch.div(i, P, rounding_mode="floor").clamp(max=s["table"].shape[1] - 1)].long().clamp(min=0)
    had = s["had"].float()
    coded = (i < enc[:, None])[:, None, :, None]

    def cached(packed, norms, win):
        v = packed[page, :, i % P].transpose(1, 2)  # [B, H, L, 96]
        v = s["cb8"].index_select(0, _codes(v).reshape(-1)).reshape(B, H, L, D) @ had
        v *= norms.view(torch.float16)[page, :, i % P].transpose(1, 2).float().unsqueeze(-1) / D
        if R:
            v = torch.where(coded, v, win[:, :, i % R].float())
        return v

    n = s["max_new"]
    b, j = _token_rows(s["cu"], T)
    q = torch.zeros(B, n, H, G, D, device="cuda")
    q[b, j] = Q.float().reshape(T, H, G, D)
    q = q.permute(0, 2, 3, 1, 4).reshape(B, H, G * n, D)
    k = cached(s["kp"], s["kn"], s["kwin"])
    scores = (q @ k.transpose(-1, -2)).div_(math.sqrt(D)).reshape(B, H, G, n, L)
    del k, q
    seen = i <= past[:, None, None] + torch.arange(n, device="cuda")[:, None]
    scores.masked_fill_(~seen[:, None, None], -math.inf)
    scores -= scores.amax(-1, keepdim=True)
    scores.exp_()
    scores /= scores.sum(-1, keepdim=True)
    v = cached(s["vp"], s["vn"], s["vwin"])
    v.masked_fill_(~(i < total[:, None])[:, None, :, None], 0)
    o = (scores.reshape(B, H, G * n, L) @ v).reshape(B, H, G, n, D)
    s["out"].copy_(o.permute(0, 3, 1, 2, 4)[b, j].reshape(T, H * G, D))
    return s["out"]


# ------------------------------------------------------------------ from the definition, in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    if s["op"] == "tables":
        return _exact_tables(s)
    if s["op"] == "append":
        return _exact_append(s)
    return _exact_attend(s)


def _exact_tables(s):
    P, R = s["P"], s["R"]
    table, free = s["table"].tolist(), s["free"].tolist()[: int(s["n_free"])]
    cu, slots = [0], []
    for b, (p, n) in enumerate(zip(s["past"], s["new"])):
        for i in range(_pages(p, P, R), _pages(p + n, P, R)):
            table[b][i] = free.pop()
        for i in range(p - R, p + n - R):
            slots.append(-1 if i < 0 else table[b][i // P] * P + i % P)
        cu.append(cu[-1] + n)
    slots += [-1] * (s["T"] - len(slots))
    return dict(table=_ints(table), cu=_ints(cu), slots=_ints(slots, torch.int64), n_free=_ints([len(free)]))


def _butterflies(x):
    """The 256-point +-1 Hadamard transform of the last axis, by sums and differences."""
    h = 1
    while h < D:
        y = x.reshape(*x.shape[:-1], D // (2 * h), 2, h)
        x = torch.stack([y[..., 0, :] + y[..., 1, :], y[..., 0, :] - y[..., 1, :]], -2).reshape(x.shape)
        h *= 2
    return x


def _exact_append(s):
    P, R, H = s["P"], s["R"], s["H"]
    c = s["cb8"].double()
    for x, packed, norms, win in ((s["K"], s["kp"], s["kn"], s["kwin"]), (s["V"], s["vp"], s["vn"], s["vwin"])):
        done = 0
        for b, (p, n) in enumerate(zip(s["past"], s["new"])):
            mine = x[done:done + n].transpose(0, 1)  # [H, n, 256]
            done += n
            if R:
                kept = [i % R for i in range(max(0, p - R), p)]
                everything = torch.cat([win[b][:, kept], mine], 1)
            else:
                everything = mine
            first = max(0, p - R)
            go = _enc(p + n, R) - first
            if go > 0:
                v = everything[:, :go].double()
                length = v.square().sum(-1).sqrt()
                y = _butterflies(v) / torch.where(length > 0, length, 1.0)[..., None]
                code = (y[..., None, :] > ((c[1:] + c[:-1]) / 2)[:, None]).sum(-2)
                bits = ((code[..., None] >> torch.arange(3, device="cuda")) & 1).reshape(H, go, NBYTES, 8)
                byte = (bits << torch.arange(8, device="cuda")).sum(-1).to(torch.uint8)
                tok = torch.arange(first, first + go, device="cuda")
                page = s["table"][b].long()[tok // P]
                packed[page, :, tok % P] = byte.transpose(0, 1)
                norms.view(torch.float16)[page, :, tok % P] = _half(length).transpose(0, 1)
            if R:
                last = min(n, R)
                where = torch.tensor([i % R for i in range(p + n - last, p + n)], dtype=torch.long, device="cuda")
                win[b][:, where] = mine[:, n - last:]
    return _cache_out(s)


def _exact_attend(s):
    P, R, H, G = s["P"], s["R"], s["H"], s["G"]
    c = s["cb8"].double()
    out = torch.zeros(s["Q"].shape, dtype=torch.float64, device="cuda")
    done = 0
    shift = torch.arange(3 * D, device="cuda")

    def vectors(packed, norms, win, b, h, e, total):
        tok = torch.arange(e, device="cuda")
        page = s["table"][b].long()[tok // P]
        rows = packed[page, h, tok % P]
        bits = (rows[:, shift // 8].to(torch.int16) >> (shift % 8)) & 1
        code = bits[:, 0::3] + 2 * bits[:, 1::3] + 4 * bits[:, 2::3]
        v = _butterflies(c[code.long()]) * (norms.view(torch.float16)[page, h, tok % P].double() / D)[:, None]
        if total > e:
            v = torch.cat([v, win[b, h][torch.arange(e, total, device="cuda") % R].double()], 0)
        return v

    for b, (p, n) in enumerate(zip(s["past"], s["new"])):
        e = _enc(p + n, R)
        ahead = torch.arange(p + n, device="cuda")[None] > (p + torch.arange(n, device="cuda"))[:, None]
        for h in range(H):
            k = vectors(s["kp"], s["kn"], s["kwin"], b, h, e, p + n)
            v = vectors(s["vp"], s["vn"], s["vwin"], b, h, e, p + n)
            for g in range(h * G, (h + 1) * G):
                a = s["Q"][done:done + n, g].double() @ k.T / 16
                a = torch.softmax(a.masked_fill(ahead, -math.inf), -1)
                out[done:done + n, g] = a @ v
        done += n
    return out

"""The int8 key/value cache operators as they are measured: appending to the paged cache, reading it back, and the
attention over it.

A cache holds keys and values as int8 codes, with one fp32 scale for each page of tokens and each head:

    k, v               int8 [pages, heads, page, dim]     codes, value = code * scale
    k_scale, v_scale   fp32 [pages, heads]

A batch of `seqs` sequences has its new tokens packed one sequence after another (`q_start`, seqs + 1 numbers); the last
n = q_start[s + 1] - q_start[s] of the kv_len[s] tokens of sequence s are the new ones, and `table[s, i]` is the page that
holds its tokens i * page .. i * page + page - 1.

Case keys: kind, dtype, seqs, heads (of keys and values), group (query heads for each of them), dim, page, q (new tokens of
the longest chunk), kv (tokens of the longest sequence, the new ones among them), spread (how much shorter the other
sequences are, 0 to 1), rot (rotated dims of a head, 0: none), interleaved (the rotation's pairs), causal, window (0: none).
"""
import math

import torch

own = False

DTYPES = {"float16": torch.float16, "bfloat16": torch.bfloat16}


def _case(name, kind, dtype, seqs, heads, group, dim, page, q, kv, spread=0.0, rot=0, interleaved=False, causal=True, window=0):
    return dict(name=name, kind=kind, dtype=dtype, seqs=seqs, heads=heads, group=group, dim=dim, page=page, q=q, kv=kv,
                spread=spread, rot=rot, interleaved=interleaved, causal=causal, window=window)


def listed():
    return [
        # one generation step of a 7B layer: eight sequences get one token each (then the pages it touched are read back)
        _case("append_decode_7b", "append", "float16", 8, 32, 1, 128, 64, 1, 1000, 0.6, 128),
        # the same of a server with grouped heads and many sequences, small pages
        _case("append_decode_70b_256", "append", "bfloat16", 256, 8, 8, 128, 16, 1, 2048, 0.8, 128),
        # chunks of seven prompts of odd lengths that go on inside a page, half of each head rotated in neighbouring pairs
        _case("append_chunks_13b", "append", "bfloat16", 7, 40, 1, 128, 32, 1021, 2500, 0.5, 64, True),
        # one short prefix read back, small heads
        _case("read_prefix", "read", "float16", 1, 8, 1, 64, 16, 333, 333),
        # four long sequences moved out of the cache
        _case("read_long_70b", "read", "bfloat16", 4, 8, 8, 128, 64, 8191, 8191, 0.3),
        # one user's generation step at a short context, as many key heads as query heads
        _case("decode_7b_single", "attention", "float16", 1, 32, 1, 128, 64, 1, 777, 0.0, 128),
        # sixteen sequences of mixed lengths of a 13B layer
        _case("decode_13b_16", "attention", "float16", 16, 40, 1, 128, 64, 1, 4096, 0.7, 128),
        # a loaded server: 64 sequences of mixed lengths, eight query heads for each key head
        _case("decode_70b_64", "attention", "bfloat16", 64, 8, 8, 128, 64, 1, 8192, 0.7, 128),
        # one very long context
        _case("decode_70b_long", "attention", "bfloat16", 1, 8, 8, 128, 128, 1, 131071, 0.0, 128),
        # five guessed tokens of each sequence checked at once, within a sliding window, small heads and pages
        _case("verify_window", "attention", "bfloat16", 16, 8, 4, 64, 16, 5, 3000, 0.5, 64, False, True, 1024),
        # a whole 7B prompt
        _case("prefill_7b", "attention", "float16", 1, 32, 1, 128, 128, 4096, 4096, 0.0, 128),
        # chunks of four prompts over what is cached of them
        _case("chunks_70b", "attention", "bfloat16", 4, 8, 8, 128, 64, 512, 8192, 0.6, 128),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["append", "read", "attention", "attention", "attention"])
    dim = rng.choice([64, 128, 128])
    page = rng.choice([16, 32, 64, 128])
    heads, group = rng.choice([(1, 1), (2, 7), (4, 3), (8, 1), (8, 4), (8, 8), (12, 1), (32, 1), (40, 1), (3, 16), (2, 20)])
    if kind == "attention":
        q = rng.choice([1, 1, _log(rng, 2, 16), _log(rng, 17, 2048)])
        kv = max(q, _log(rng, 1, 65536 if q < 17 else 8192))
        # no more than the largest listed case: 4096 x 4096 / 2 pairs of 32 heads, and about 0.5 GB of cache
        seqs = min(_log(rng, 1, 128), (1 << 32) // (kv * heads * dim * 8) or 1, (1 << 28) // (q * kv * heads * group) or 1)
        q = min(q, max(1, (1 << 28) // (kv * heads * group)))
    else:
        q = rng.choice([1, _log(rng, 2, 4096)])
        kv = q + (0 if rng.random() < 0.3 else _log(rng, 1, 4096))
        seqs = max(1, min(_log(rng, 1, 256), (1 << 25) // (max(q, page) * heads * dim), (1 << 28) // (kv * heads * dim)))
    rot = rng.choice([0, dim // 2, dim, dim])
    c = _case("", kind, rng.choice(["float16", "bfloat16"]), max(1, seqs), heads, group, dim, page, q, kv, round(rng.random(), 3),
              rot, rng.random() < 0.4, rng.random() < 0.8, rng.choice([0, 0, _log(rng, 1, 4096)]))
    del c["name"]
    return c


def _lengths(c):
    """(new tokens, tokens) of each sequence, the first the longest: a part of the case, the same for every seed."""
    ns, ls = [], []
    for s in range(c["seqs"]):
        f = 1.0 - c["spread"] * ((s * 0.6180339887) % 1.0)
        n = max(1, int(c["q"] * f))
        ns.append(n)
        ls.append(max(n, int(c["kv"] * f)))
    return ns, ls


def _starts(ns):
    out = [0]
    for n in ns:
        out.append(out[-1] + n)
    return out


def prepare(case, seed):
    c, dev = case, "cuda"
    g = torch.Generator(device=dev).manual_seed(seed)
    dt, H, D, page, S = DTYPES[c["dtype"]], c["heads"], c["dim"], c["page"], c["seqs"]
    ns, ls = _lengths(c)
    used = [-(-n // page) for n in ls]
    width = max(used)
    pages = sum(used) + 1                                    # page 0 is nobody's
    order = torch.randperm(pages - 1, generator=torch.Generator().manual_seed(seed)) + 1
    table = torch.zeros((S, width), dtype=torch.int32)
    at = 0
    for s in range(S):
        table[s, :used[s]] = order[at:at + used[s]].to(torch.int32)
        at += used[s]

    def stored(std):
        # a few channels are several times larger than the rest, as in trained models' keys
        gain = torch.ones(D, device=dev)
        gain[torch.randperm(D, generator=g, device=dev)[:4]] = 3.0
        codes = torch.empty((pages, H, page, D), dtype=torch.int8, device=dev)
        scale = torch.empty((pages, H), dtype=torch.float32, device=dev)
        step = max(1, (1 << 27) // (H * page * D))
        for p in range(0, pages, step):
            x = torch.randn((min(step, pages - p), H, page, D), generator=g, device=dev) * (gain * std)
            m = x.abs().amax(dim=(2, 3)) / 127
            scale[p:p + step] = m
            codes[p:p + step] = torch.round(x / m[:, :, None, None]).to(torch.int8)
        return codes, scale

    k, k_scale = stored(1.0)
    v, v_scale = stored(0.5)
    T = sum(ns)
    st = dict(case=c, tokens=T, max_q=max(ns), max_kv=max(ls), dtype=dt, k=k, v=v, k_scale=k_scale, v_scale=v_scale,
              q_start=torch.tensor(_starts(ns), dtype=torch.int32, device=dev),
              kv_len=torch.tensor(ls, dtype=torch.int32, device=dev), table=table.to(dev))
    st["cos"] = st["sin"] = None
    if c["rot"]:
        i = torch.arange(c["rot"] // 2, device=dev, dtype=torch.float64)
        ang = torch.arange(max(ls), device=dev, dtype=torch.float64)[:, None] * (10000.0 ** (-2.0 * i / c["rot"]))
        st["cos"], st["sin"] = ang.cos().float(), ang.sin().float()
    if c["kind"] == "append":
        # keys and values as a fused projection leaves them: rows of one matrix
        Hq = H * c["group"]
        qkv = torch.randn((T, (Hq + 2 * H) * D), generator=g, device=dev).to(dt)
        st["K"] = qkv[:, Hq * D:(Hq + H) * D].view(T, H, D)
        st["V"] = qkv[:, (Hq + H) * D:].view(T, H, D)
        # what is read back: from the first token of the first page that the new tokens touch
        back = [l - (l - n) // page * page for n, l in zip(ns, ls)]
        st["back_start"] = torch.tensor(_starts(back), dtype=torch.int32, device=dev)
        st["back_tokens"], st["back_max"] = sum(back), max(back)
    elif c["kind"] == "attention":
        st["Q"] = (torch.randn((T, H * c["group"], D), generator=g, device=dev) * 1.5).to(dt)
    if own:
        # a serving program keeps these for as long as the tensors behind them
        import int8_matmul_amd as li8
        st["cache"] = li8.KVCache(k, v, k_scale, v_scale)
        st["batch"] = li8.KVBatch(st["q_start"], st["kv_len"], st["table"], T, max(ns), max(ls))
        st["rope"] = li8.Rope(st["cos"], st["sin"], c["interleaved"]) if c["rot"] else None
        if c["kind"] == "append":
            st["back"] = li8.KVBatch(st["back_start"], st["kv_len"], st["table"], st["back_tokens"], st["back_max"], max(ls))
        if c["kind"] == "attention":
            st["workspace"] = li8.new_kv_attention_workspace(st["batch"], st["cache"], H * c["group"])
    return st


def run(st):
    c = st["case"]
    if own:
        import int8_matmul_amd as li8
        if c["kind"] == "append":
            li8.kv_append(st["K"], st["V"], st["cache"], st["batch"], rope=st["rope"])
            k, v = li8.kv_read(st["cache"], st["back"], st["dtype"])
            return {"k": k, "v": v, "k_scale": st["k_scale"], "v_scale": st["v_scale"]}
        if c["kind"] == "read":
            k, v = li8.kv_read(st["cache"], st["batch"], st["dtype"])
            return {"k": k, "v": v}
        return li8.kv_attention(st["Q"], st["cache"], st["batch"], scale=1.0 / math.sqrt(c["dim"]), rope=st["rope"],
                                causal=c["causal"], window=c["window"], workspace=st["workspace"])
    if c["kind"] == "append":
        _append(st)
        k, v = _read(st, st["back_start"], st["back_tokens"])
        return {"k": k, "v": v, "k_scale": st["k_scale"], "v_scale": st["v_scale"]}
    if c["kind"] == "read":
        k, v = _read(st, st["q_start"], st["tokens"])
        return {"k": k, "v": v}
    return _attention(st)


# ---- the plain forms ----

def _rotate(x, pos, st):
    """Rotation of x [..., heads, dim] (fp32) by the table's rows pos [...]."""
    c = st["case"]
    if not c["rot"]:
        return x
    R = c["rot"]
    cos, sin = st["cos"][pos][..., None, :], st["sin"][pos][..., None, :]
    y = x.clone()
    if c["interleaved"]:
        a, b = x[..., 0:R:2], x[..., 1:R:2]
        y[..., 0:R:2] = a * cos - b * sin
        y[..., 1:R:2] = b * cos + a * sin
    else:
        a, b = x[..., :R // 2], x[..., R // 2:R]
        y[..., :R // 2] = a * cos - b * sin
        y[..., R // 2:R] = b * cos + a * sin
    return y


def _append(st):
    c = st["case"]
    page, S, T = c["page"], c["seqs"], st["tokens"]
    n = (st["q_start"][1:] - st["q_start"][:-1]).long()
    L = st["kv_len"].long()
    first = (L - n) // page
    touched = (st["max_q"] + page - 2) // page + 1
    b = first[:, None] + torch.arange(touched, device=L.device)                     # [S, touched] page of the sequence
    live = b * page < L[:, None]
    # pages that the sequence does not have are the null page, whose contents go back as they were
    ids = torch.where(live, st["table"].long().gather(1, b.clamp(max=st["table"].shape[1] - 1)), 0)
    pos = b[:, :, None] * page + torch.arange(page, device=L.device)                # [S, touched, page]
    begin = (L - n)[:, None, None]
    new = live[:, :, None] & (pos >= begin) & (pos < L[:, None, None])
    old = live[:, :, None] & (pos < begin)
    row = (st["q_start"][:-1].long()[:, None, None] + pos - begin).clamp(0, T - 1)
    newr, oldr = new[:, :, None, :, None], old[:, :, None, :, None]
    for x, codes, scale, rotated in ((st["K"], st["k"], st["k_scale"], True), (st["V"], st["v"], st["v_scale"], False)):
        x = x.float()[row]                                                          # [S, touched, page, H, D]
        if rotated:
            x = _rotate(x, pos.clamp(0, st["max_kv"] - 1), st)
        x = x.permute(0, 1, 3, 2, 4)
        before, s_before = codes[ids], scale[ids]
        amax = torch.where(newr, x.abs(), 0.0).amax(dim=(3, 4))
        s_old = torch.where(old.any(2)[:, :, None], s_before, 0.0)
        s = torch.maximum(s_old, amax / 127)
        r = torch.where(s > 0, 1.0 / s, 0.0).clamp(max=3.4028234663852886e38)[..., None, None]
        fresh = torch.round(x * r).clamp(-127, 127)
        kept = before.float()
        moved = torch.round(kept * s_old[..., None, None] * r).clamp(-127, 127)
        kept = torch.where(oldr & (s > s_old)[..., None, None], moved, kept)
        codes[ids] = torch.where(newr, fresh, kept).to(torch.int8)
        scale[ids] = torch.where(live[:, :, None], s, s_before)


def _read(st, start, tokens):
    page = st["case"]["page"]
    t = torch.arange(tokens, device=start.device)
    s = torch.bucketize(t, start[1:].long(), right=True)
    pos = (st["kv_len"].long()[s] - start[1:].long()[s]) + t
    p = st["table"].long()[s, pos // page]
    return tuple((codes[p, :, pos % page].float() * scale[p][:, :, None]).to(st["dtype"])
                 for codes, scale in ((st["k"], st["k_scale"]), (st["v"], st["v_scale"])))


def _attention(st):
    c = st["case"]
    S, H, G, D, T, mq = c["seqs"], c["heads"], c["group"], c["dim"], st["tokens"], st["max_q"]
    dev = st["Q"].device
    n = (st["q_start"][1:] - st["q_start"][:-1]).long()
    L = st["kv_len"].long()
    ids = st["table"].long()
    k, v = ((codes[ids].float() * scale[ids][..., None, None]).permute(0, 2, 1, 3, 4).reshape(S, H, -1, D)
            for codes, scale in ((st["k"], st["k_scale"]), (st["v"], st["v_scale"])))
    i = torch.arange(mq, device=dev)
    pos = (L - n)[:, None] + i                                                      # [S, mq]
    q = st["Q"].float()[(st["q_start"][:-1].long()[:, None] + i).clamp(max=T - 1)]  # [S, mq, Hq, D]
    q = _rotate(q, pos.clamp(0, st["max_kv"] - 1), st)
    q = q.reshape(S, mq, H, G, D).permute(0, 2, 3, 1, 4).reshape(S, H, G * mq, D)
    s = torch.matmul(q, k.transpose(2, 3).contiguous()) * (1.0 / math.sqrt(D))
    t = torch.arange(k.shape[2], device=dev)
    seen = (t < L[:, None, None]).expand(S, mq, -1)
    if c["causal"]:
        seen = seen & (t <= pos[:, :, None])
    if c["window"]:
        seen = seen & (t > pos[:, :, None] - c["window"])
    s = s.view(S, H, G, mq, -1).masked_fill_(~seen[:, None, None], -math.inf)
    m = s.amax(dim=-1, keepdim=True).clamp(min=-3.0e38)
    p = torch.exp(s - m)
    total = p.sum(dim=-1, keepdim=True)
    o = torch.matmul(p.view(S, H, G * mq, -1), v).view(S, H, G, mq, D)
    o = torch.where(total > 0, o / total, 0.0).permute(0, 3, 1, 2, 4).reshape(S, mq, H * G, D)
    tok = torch.arange(T, device=dev)
    seq = torch.bucketize(tok, st["q_start"][1:].long(), right=True)
    return o[seq, tok - st["q_start"].long()[seq]].to(st["dtype"])


# ---- how much work ----

def work(case):
    c = case
    ns, ls = _lengths(c)
    H, D, page, T = c["heads"], c["dim"], c["page"], sum(ns)
    row = H * D
    if c["kind"] == "read":
        return {"bytes": 2 * T * row * (1 + 2), "flops": 2 * T * row}
    if c["kind"] == "append":
        back = sum(l - (l - n) // page * page for n, l in zip(ns, ls))
        return {"bytes": 2 * T * row * (2 + 1) + 2 * back * row * (1 + 2) + 4 * T * c["rot"],
                "flops": 2 * T * row * 4 + 2 * back * row}
    w, kv, pairs = c["window"], 0, 0
    for n, l in zip(ns, ls):
        kv += l - (max(0, l - n + 1 - w) if w else 0)
        for i in range(n):
            p = l - n + i
            pairs += (p + 1 if c["causal"] else l) - (max(0, p + 1 - w) if w else 0)
    Hq = H * c["group"]
    return {"bytes": 2 * kv * row + 8 * (kv // page + 1) * H + 2 * 2 * T * Hq * D + 4 * T * c["rot"], "flops": 4 * pairs * Hq * D}


# ---- the same from the definitions, in 64 bits, one sequence after another ----

def exact(case, seed):
    c = case
    st = prepare(case, seed)
    ns, ls = _lengths(c)
    table = st["table"].tolist()
    page, H, G, D, R = c["page"], c["heads"], c["group"], c["dim"], c["rot"]
    f64 = torch.float64

    def turn(x, p0):
        """Rows x [n, heads, D] at positions p0, p0 + 1, ... as complex numbers times cos + i sin."""
        if not R:
            return x
        z = torch.complex(st["cos"][p0:p0 + len(x)].to(f64), st["sin"][p0:p0 + len(x)].to(f64))[:, None]
        head, tail = x[..., :R], x[..., R:]
        if c["interleaved"]:
            w = torch.view_as_complex(head.reshape(*head.shape[:-1], R // 2, 2).contiguous()) * z
            head = torch.view_as_real(w).reshape(head.shape)
        else:
            w = torch.complex(head[..., :R // 2].contiguous(), head[..., R // 2:].contiguous()) * z
            head = torch.cat([w.real, w.imag], dim=-1)
        return torch.cat([head, tail], dim=-1)

    def held(codes, scale, s, first, last):
        """Values of the tokens first .. last - 1 of sequence s, [tokens, heads, D]."""
        a, b = first // page, -(-last // page)
        ids = torch.tensor(table[s][a:b], device=codes.device)
        x = codes[ids].to(f64) * scale[ids].to(f64)[:, :, None, None]
        return x.transpose(1, 2).reshape(-1, H, D)[first - a * page:last - a * page]

    starts = _starts(ns)
    if c["kind"] == "read":
        return {n: torch.cat([held(st[n], st[n + "_scale"], s, ls[s] - ns[s], ls[s]) for s in range(c["seqs"])]) for n in ("k", "v")}
    if c["kind"] == "append":
        out = {}
        for name, src in (("k", "K"), ("v", "V")):
            scales, values = st[name + "_scale"].to(f64), []
            for s in range(c["seqs"]):
                begin = ls[s] - ns[s]
                x = st[src][starts[s]:starts[s + 1]].to(f64)
                x = turn(x, begin) if name == "k" else x
                for b in range(begin // page, -(-ls[s] // page)):
                    lo, hi = max(begin, b * page), min(ls[s], (b + 1) * page)
                    rows = x[lo - begin:hi - begin]
                    need, p = rows.abs().amax(dim=(0, 2)) / 127, table[s][b]
                    if lo > b * page:
                        kept = st[name][p, :, :lo - b * page].transpose(0, 1).to(f64) * scales[p][:, None]
                        scale = torch.maximum(need, scales[p])
                        kept = torch.round(kept / scale[:, None])
                        rows = torch.cat([kept, torch.round(rows / scale[:, None])])
                    else:
                        scale = need
                        rows = torch.round(rows / scale[:, None])
                    scales[p] = scale
                    values.append(rows * scale[:, None])
            out[name], out[name + "_scale"] = torch.cat(values), scales
        return out
    outs = []
    for s in range(c["seqs"]):
        n, l = ns[s], ls[s]
        begin = l - n
        first = max(0, begin + 1 - c["window"]) if c["window"] else 0
        k, v = (held(st[x], st[x + "_scale"], s, first, l).transpose(0, 1) for x in ("k", "v"))      # [H, l - first, D]
        step = max(1, (1 << 28) // (H * G * (l - first)))
        for i in range(0, n, step):
            q = turn(st["Q"][starts[s] + i:starts[s] + min(n, i + step)].to(f64), begin + i)
            m = len(q)
            q = q.reshape(m, H, G, D).permute(1, 0, 2, 3).reshape(H, m * G, D)
            z = torch.matmul(q, k.transpose(1, 2).contiguous()) / math.sqrt(D)
            at = torch.arange(begin + i, begin + i + m, device=z.device).repeat_interleave(G)[:, None]
            key = torch.arange(first, l, device=z.device)[None]
            hide = torch.zeros((m * G, l - first), dtype=torch.bool, device=z.device)
            if c["causal"]:
                hide |= key > at
            if c["window"]:
                hide |= key <= at - c["window"]
            z = torch.softmax(z.masked_fill(hide, -math.inf), dim=-1).nan_to_num(0.0)
            outs.append(torch.matmul(z, v).reshape(H, m, G, D).permute(1, 0, 2, 3).reshape(m, H * G, D))
    return torch.cat(outs)

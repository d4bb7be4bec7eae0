"""What is timed of the 4-bit decoding operators, and their plain forms.

Four operators that a server needs to generate tokens on rotated 4-bit
weights and a rotated 4-bit cache of keys and values:

  matvec     a few tokens times packed INT4 weights with one scale per group
             of channels (convrot_w4g_linear)
  attention  queries of the newest tokens over a paged INT4 cache of keys and
             values (convrot_kv4_attention)
  append     new keys and values into that cache, and the rows read back
             (convrot_kv4_append, convrot_kv4_read)
  plan       block table, slot map and positions of a step from the request
             lengths (convrot_kv4_plan)

``run`` computes them with elementary torch operations, or with the package's
kernels where ``own`` is true.
"""
import math

import torch

own = False

# Codes are 4-bit two's complement in [-7, 7], two per byte, low nibble first.


def listed():
    """The timed cases; each comment says what it stands for."""
    return [
        # the smallest projection of the layer workloads, one token: launch latency counts
        dict(name="matvec 1x1024-1024", op="matvec", tokens=1, K=1024, N=1024, group=256, scale_group=64, bias=True),
        # one decoding request through the up projection of the skinny workloads
        dict(name="matvec 1x4096-14336", op="matvec", tokens=1, K=4096, N=14336, group=64, scale_group=64, bias=False),
        # a decoding batch of 16 through the same layer, coarser scales
        dict(name="matvec 16x4096-14336", op="matvec", tokens=16, K=4096, N=14336, group=64, scale_group=128, bias=False),
        # a long, odd-sized down projection on rows that are rotated already, the finest scales
        dict(name="matvec 5x12288-8197", op="matvec", tokens=5, K=12288, N=8197, group=0, scale_group=32, bias=True),
        # one request with a short history: latency counts
        dict(name="attention 1x1021", op="attention", requests=1, queries=1, heads=32, kv_heads=8, head_dim=128,
             group=64, page=16, shortest=1021, longest=1021),
        # a full decoding batch of ragged histories: the cache's bytes count
        dict(name="attention 64x8192", op="attention", requests=64, queries=1, heads=32, kv_heads=8, head_dim=128,
             group=64, page=64, shortest=1500, longest=8192),
        # two requests with very long histories: the length has to be split
        dict(name="attention 2x131072", op="attention", requests=2, queries=1, heads=64, kv_heads=8, head_dim=128,
             group=64, page=64, shortest=100003, longest=131072),
        # several drafted tokens a request to be verified, wide heads, a few shared heads
        dict(name="attention 16x5x3000", op="attention", requests=16, queries=5, heads=16, kv_heads=4, head_dim=256,
             group=256, page=32, shortest=300, longest=3001),
        # the new token of each of 64 decoding requests
        dict(name="append 64", op="append", tokens=64, kv_heads=8, head_dim=128, group=64, page=16, scattered=True),
        # the prompts of a prefill step
        dict(name="append 16384", op="append", tokens=16384, kv_heads=8, head_dim=128, group=64, page=64, scattered=False),
        # a decoding step of 64 requests
        dict(name="plan 64x1", op="plan", requests=64, page=16, cached=8192, new=1, padding=0),
        # a large mixed step: prompts of up to 300 tokens, finished requests, padding of a captured graph
        dict(name="plan 1024x300", op="plan", requests=1024, page=16, cached=4096, new=300, padding=1000),
    ]


def _log(rng, low, high):
    """A whole number of low .. high, even over the logarithm."""
    return min(high, max(low, int(round(math.exp(rng.uniform(math.log(low), math.log(high + 1)))))))


def draw(rng):
    """One more case of the same ranges."""
    op = rng.choice(["matvec", "matvec", "attention", "attention", "append", "plan"])
    if op == "matvec":
        group = rng.choice([0, 64, 256])
        step = max(64, group, scale_group := rng.choice([32, 64, 128]))
        return dict(op=op, tokens=_log(rng, 1, 32), K=step * _log(rng, 1, 12288 // step), N=_log(rng, 1, 14336),
                    group=group, scale_group=scale_group, bias=rng.random() < 0.5)
    if op == "attention":
        head_dim = rng.choice([64, 128, 128, 256])
        requests, kv_heads = _log(rng, 1, 64), rng.choice([1, 2, 4, 8])
        longest = _log(rng, 1, min(131072, (64 * 8192 * 8 * 128) // (2 * requests * kv_heads * head_dim)))
        return dict(op=op, requests=requests, queries=rng.choice([1, 1, 1, 2, 3, 5, 8]),
                    heads=kv_heads * rng.choice([1, 2, 3, 4, 7, 8, 16]), kv_heads=kv_heads, head_dim=head_dim,
                    group=256 if head_dim == 256 and rng.random() < 0.5 else 64, page=rng.choice([16, 32, 64, 128, 256]),
                    shortest=_log(rng, 1, longest), longest=longest)
    if op == "append":
        head_dim = rng.choice([64, 128, 256])
        return dict(op=op, tokens=_log(rng, 1, 8192), kv_heads=rng.choice([1, 2, 3, 4, 8]), head_dim=head_dim,
                    group=256 if head_dim == 256 and rng.random() < 0.5 else 64, page=rng.choice([16, 32, 64, 128, 256]),
                    scattered=rng.random() < 0.5)
    return dict(op=op, requests=_log(rng, 1, 1024), page=rng.choice([16, 32, 64, 128, 256]), cached=_log(rng, 1, 4096),
                new=_log(rng, 1, 256), padding=rng.choice([0, 1, 500]))


# ------------------------------------------------------------------ sizes of a case

def _spread(low, high, count):
    """`count` lengths from low to high, even over the logarithm."""
    if count == 1:
        return [high]
    return [int(round(low * (high / low) ** (i / (count - 1)))) for i in range(count)]


def _queries(case):
    """New tokens a request: every third request brings about half of them."""
    q = case["queries"]
    return [q - (q // 2 if b % 3 == 2 else 0) for b in range(case["requests"])]


def _plan_new(case):
    """New tokens a request of a plan: prompts of many lengths between single
    tokens; every seventeenth request is finished (-1)."""
    return [-1 if b % 17 == 16 else 1 + (case["new"] - 1) * ((b * 7) % 11) // 10 for b in range(case["requests"])]


def work(case):
    """Bytes and floating-point operations that one pass cannot do without."""
    op = case["op"]
    if op == "matvec":
        M, K, N = case["tokens"], case["K"], case["N"]
        return {"bytes": N * K // 2 + 2 * N * K // case["scale_group"] + 2 * M * K + 2 * M * N + 2 * N * case["bias"],
                "flops": 2 * M * N * K + (2 * M * K * int(math.log2(case["group"])) if case["group"] else 0)}
    if op == "attention":
        H, D = case["kv_heads"], case["head_dim"]
        lens, new = _spread(case["shortest"], case["longest"], case["requests"]), _queries(case)
        rows = sum(lens) * H
        return {"bytes": rows * (D + 4) + 4 * sum(new) * case["heads"] * D + sum(-(-n // case["page"]) * 4 for n in lens),
                "flops": sum(4 * n * q for n, q in zip(lens, new)) * case["heads"] * D}
    if op == "append":
        rows = case["tokens"] * case["kv_heads"] * 2
        # keys and values in, codes and scales out and in again, rows out
        return {"bytes": rows * (2 * case["head_dim"] + 2 * (case["head_dim"] // 2 + 2) + 2 * case["head_dim"]) + 16 * case["tokens"],
                "flops": rows * case["head_dim"] * (4 * int(math.log2(case["group"])) + 6)}
    new = _plan_new(case)
    tokens = sum(n for n in new if n > 0)
    pages = tokens // case["page"] + case["requests"] // 2
    return {"bytes": 12 * (tokens + case["padding"]) + 8 * pages + 16 * case["requests"], "flops": 0}


# ------------------------------------------------------------------ inputs

def _normal_codes(shape, g):
    """Packed codes as rotated, rowwise scaled rows have them: near normal,
    the row's largest value at 7."""
    u = torch.empty(*shape, 2, dtype=torch.bfloat16, device="cuda").normal_(0.0, 2.6, generator=g)
    c = u.round_().clamp_(-7, 7).to(torch.int8)
    return ((c[..., 1] << 4) | (c[..., 0] & 15)).view(torch.uint8)


def _scales(shape, low, high, g):
    return torch.empty(shape, dtype=torch.float32, device="cuda").uniform_(low, high, generator=g).to(torch.bfloat16)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    op = case["op"]
    s = dict(case)
    if op == "matvec":
        M, K, N = case["tokens"], case["K"], case["N"]
        x = torch.empty(M, K, dtype=torch.float32, device="cuda").normal_(generator=g)
        # a few channels are far larger than the others, as a model's activations have them
        x[:, torch.randperm(K, generator=g, device="cuda")[:max(1, K // 100)]] *= 20.0
        s["x"] = x.to(torch.bfloat16)
        s["qw"] = _normal_codes((N, K // 2), g)
        s["sg"] = _scales((N, K // case["scale_group"]), 0.004, 0.012, g)
        s["b"] = torch.empty(N, device="cuda").normal_(0, 0.02, generator=g).to(torch.bfloat16) if case["bias"] else None
        return s
    if op == "plan":
        return _prepare_plan(case, g, s)
    H, D, page = case["kv_heads"], case["head_dim"], case["page"]
    if op == "append":
        T = case["tokens"]
        pages = (T if case["scattered"] else -(-T // page)) + 3
        at = torch.randperm(pages, generator=g, device="cuda")
        t = torch.arange(T, device="cuda")
        if case["scattered"]:   # one token of each request, anywhere in its last page
            s["slots"] = at[t] * page + torch.randint(page, (T,), generator=g, device="cuda")
        else:                   # one run of tokens that begins inside a page
            u = t + page // 3
            s["slots"] = at[u // page] * page + u % page
        # keys and values are columns of the fused projection's rows
        qkv = torch.empty(T, 4 * H * D, dtype=torch.bfloat16, device="cuda").normal_(generator=g)
        s["k"] = qkv[:, 2 * H * D:3 * H * D].unflatten(1, (H, D))
        s["v"] = qkv[:, 3 * H * D:].unflatten(1, (H, D))
        s["cache"] = tuple(torch.zeros(pages, H, page, *w, dtype=d, device="cuda")
                           for w, d in (((D // 2,), torch.uint8), ((), torch.bfloat16)) * 2)
        return s
    order = torch.randperm(case["requests"], generator=g, device="cuda")
    lens = torch.tensor(_spread(case["shortest"], case["longest"], case["requests"]), device="cuda")[order]
    new = torch.tensor(_queries(case), device="cuda")
    most = -(-case["longest"] // page)
    pages = case["requests"] * most
    s["cache"] = tuple(f() for f in (lambda: _normal_codes((pages, H, page, D // 2), g),
                                     lambda: _scales((pages, H, page), 0.3, 0.5, g)) * 2)
    s["table"] = torch.randperm(pages, generator=g, device="cuda").view(case["requests"], most).int()
    s["lens"] = lens.int()
    s["cu_q"] = torch.cat([torch.zeros(1, dtype=torch.int64, device="cuda"), new.cumsum(0)]).int()
    s["q"] = torch.empty(sum(_queries(case)), case["heads"], D, device="cuda").normal_(0, 1.5, generator=g).to(torch.bfloat16)
    s["scale"] = D ** -0.5
    return s


def _prepare_plan(case, g, s):
    B, page = case["requests"], case["page"]
    new = _plan_new(case)
    order = torch.randperm(B, generator=g, device="cuda")
    s["new"] = torch.tensor(new, device="cuda")[order].int()
    s["cached"] = torch.randint(case["cached"] + 1, (B,), generator=g, device="cuda").int()
    most = -(-(case["cached"] + case["new"]) // page)
    spare = sum(-(-max(n, 0) // page) + 1 for n in new)
    pages = torch.randperm(B * most + spare, generator=g, device="cuda").int()
    s["table"] = pages[:B * most].view(B, most).clone()
    s["free"] = pages[B * most:].repeat(2)[:spare + B * most].contiguous()   # room for pages that come back
    if s["free"].numel() < spare + B * most:
        s["free"] = torch.cat([s["free"], s["free"].new_zeros(spare + B * most - s["free"].numel())])
    s["count"] = torch.tensor([spare], dtype=torch.int32, device="cuda")
    s["capacity"] = sum(max(n, 0) for n in new) + case["padding"]
    return s


# ------------------------------------------------------------------ plain forms

def _hadamard(n):
    """The normalised regular Hadamard matrix of order n = 4^k."""
    t = torch.ones(4, 4, device="cuda") - 2 * torch.eye(4, device="cuda")
    h = torch.kron(t, torch.kron(t, t)) if n == 64 else torch.kron(torch.kron(t, t), torch.kron(t, t))
    return h / math.sqrt(n)


def _rotate(x, group):
    return (x.unflatten(-1, (-1, group)) @ _hadamard(group)).flatten(-2) if group else x


def _unpack(codes):
    """uint8 [..., n] -> float [..., 2 n], low nibble first."""
    both = torch.stack([codes & 15, codes >> 4], -1).flatten(-2)
    return (both ^ 8).float() - 8.0


def _plain_matvec(s):
    x = _rotate(s["x"].float(), s["group"])
    w = (_unpack(s["qw"]).unflatten(1, (-1, s["scale_group"])) * s["sg"].float()[..., None]).flatten(1)
    y = x @ w.T
    return (y if s["b"] is None else y + s["b"].float()).to(torch.bfloat16)


def _plain_attention(s):
    q, table, lens, cu = s["q"], s["table"].long().clamp(min=0), s["lens"].long(), s["cu_q"].long()
    B, H, D, page = s["requests"], s["kv_heads"], s["head_dim"], s["page"]
    nq, G, L = s["queries"], s["heads"] // s["kv_heads"], table.shape[1] * page
    kc, ks, vc, vs = s["cache"]

    def rows(codes, scales):   # [B, H, L, D], still rotated
        c = _unpack(codes[table].transpose(1, 2).reshape(B, H, L, D // 2))
        return c.mul_(scales[table].transpose(1, 2).reshape(B, H, L, 1).float())

    count = cu[1:] - cu[:-1]
    i, j = torch.arange(nq, device="cuda"), torch.arange(L, device="cuda")
    at = (cu[:-1, None] + i).clamp(max=q.shape[0] - 1)
    qr = _rotate(q.float(), s["group"])[at]                       # [B, nq, Hq, D]
    qr = qr.unflatten(2, (H, G)).permute(0, 2, 1, 3, 4).reshape(B, H, nq * G, D)
    score = (qr @ rows(kc, ks).transpose(2, 3)).mul_(s["scale"])
    seen = (j <= (lens - count)[:, None, None] + i[:, None]) & (i < count[:, None])[..., None]   # [B, nq, L]
    seen = seen[:, None, :, None, :].expand(B, 1, nq, G, L).reshape(B, 1, nq * G, L)
    score = score.masked_fill_(~seen, -math.inf)
    top = score.amax(-1, keepdim=True)
    e = (score - torch.where(top == -math.inf, torch.zeros_like(top), top)).exp_()
    total = e.sum(-1, keepdim=True)
    o = (e @ rows(vc, vs)) / torch.where(total == 0, torch.ones_like(total), total)
    o = _rotate(o, s["group"]).view(B, H, nq, G, D).permute(0, 2, 1, 3, 4).reshape(B, nq, H * G, D)
    t = torch.arange(q.shape[0], device="cuda")
    b = torch.searchsorted(cu[1:].contiguous(), t, right=True)
    return o[b, t - cu[b]].to(torch.bfloat16)


def _plain_append(s):
    kc, ks, vc, vs = s["cache"]
    page, slots = s["page"], s["slots"]
    at, off = slots // page, slots % page

    def store(x, codes, scales):
        y = _rotate(x.float(), s["group"])
        scale = (y.abs().amax(-1) / y.new_tensor(7.0)).to(torch.bfloat16)
        safe = torch.where(scale == 0, torch.ones_like(scale), scale).float()
        v = y * (1.0 / safe)[..., None]
        c = (torch.sign(v) * torch.floor(v.abs() + 0.5)).clamp_(-7, 7).to(torch.int8)
        codes[at, :, off] = ((c[..., 1::2] << 4) | (c[..., 0::2] & 15)).view(torch.uint8)
        scales[at, :, off] = scale

    def load(codes, scales):
        y = _unpack(codes[at, :, off]) * scales[at, :, off].float()[..., None]
        return _rotate(y, s["group"]).to(torch.bfloat16)

    store(s["k"], kc, ks)
    store(s["v"], vc, vs)
    return load(kc, ks), load(vc, vs)


def _plain_plan(s):
    page, table, free = s["page"], s["table"], s["free"]
    cached, new, count = s["cached"].long(), s["new"].long(), s["count"].long()
    B, most = table.shape
    zero = torch.zeros(1, dtype=torch.int64, device="cuda")
    done = new < 0
    n = new.clamp(min=0)
    have = (cached + page - 1) // page
    length = torch.where(done, torch.zeros_like(n), cached + n)
    take = torch.where(done, torch.zeros_like(n), ((length + page - 1) // page) - have)
    back = torch.where(done, have, torch.zeros_like(n))
    cu_q, cu_take, cu_back = (torch.cat([zero, v.cumsum(0)]) for v in (n, take, back))
    j = torch.arange(most, device="cuda")
    held = count + cu_back[-1:]
    # pages of finished requests go on top of the free list, the step's pages come off its top
    put = torch.where(done[:, None] & (j < have[:, None]), count + cu_back[:-1, None] + j, free.numel())
    room = torch.cat([free, free.new_zeros(1)])
    room[put.flatten()] = table.flatten()
    fits = (cu_take[-1:] <= held) & (length.amax() <= most * page) & (cu_q[-1:] <= s["capacity"]) & (held <= free.numel())
    room = torch.where(fits, room[:-1], free)
    mine = ~done[:, None] & (j >= have[:, None]) & (j < (have + take)[:, None]) & fits
    got = room[(held - 1 - (cu_take[:-1, None] + j - have[:, None])).clamp(0, free.numel() - 1)]
    table_ = torch.where(mine, got, table)
    t = torch.arange(s["capacity"], device="cuda")
    b = torch.searchsorted(cu_q[1:].contiguous(), t, right=True).clamp(max=B - 1)
    real = (t < cu_q[-1]) & fits
    pos = torch.where(real, cached[b] + t - cu_q[b], -1)
    slot = torch.where(real, table_[b, (pos // page).clamp(0, most - 1)].long() * page + pos % page, -1)
    left = torch.where(fits, held - cu_take[-1:], count)
    lens = torch.where(fits, length, cached)
    return dict(block_table=table_, free_pages=room, seq_lens=lens.int(), cu_q=torch.where(fits, cu_q, 0).int(),
                slots=slot, positions=pos.int(), free_count=left.int())


def run(s):
    op = s["op"]
    if own:
        import rotated_w4a4_quantized_b200 as cr
        if op == "matvec":
            return cr.convrot_w4g_linear(s["x"], s["qw"], s["sg"], s["b"], s["group"], s["scale_group"])
        if op == "attention":
            return cr.convrot_kv4_attention(s["q"], s["cache"], s["table"], s["lens"], s["cu_q"], s["scale"], s["group"])
        if op == "append":
            cr.convrot_kv4_append(s["k"], s["v"], s["cache"], s["slots"], s["group"])
            return cr.convrot_kv4_read(s["cache"], s["slots"], s["group"])
        p = cr.convrot_kv4_plan(s["cached"], s["new"], s["table"], s["free"], s["count"], s["page"], s["capacity"])
        return dict(block_table=s["table"], free_pages=s["free"], seq_lens=p.seq_lens, cu_q=p.cu_q, slots=p.slots,
                    positions=p.positions, free_count=p.free_count)
    return {"matvec": _plain_matvec, "attention": _plain_attention, "append": _plain_append, "plan": _plain_plan}[op](s)


# ------------------------------------------------------------------ 64 bits

def _signs(n):
    """H_n entry by entry: (-1)^(base-4 digits in which i and j agree) / sqrt(n)."""
    i = torch.arange(n, device="cuda")
    agree = torch.zeros(n, n, dtype=torch.int64, device="cuda")
    for d in range(3 if n == 64 else 4):
        digit = (i >> (2 * d)) & 3
        agree += digit[:, None] == digit[None, :]
    return (1 - 2 * (agree % 2)).double() / n ** 0.5


def _turn(y, group):
    if not group:
        return y
    shape = y.shape
    return torch.einsum("...gi,ij->...gj", y.reshape(*shape[:-1], shape[-1] // group, group), _signs(group)).reshape(shape)


def _values(codes):
    table = torch.tensor([0, 1, 2, 3, 4, 5, 6, 7, -8, -7, -6, -5, -4, -3, -2, -1], dtype=torch.float64, device="cuda")
    out = torch.empty(*codes.shape[:-1], 2 * codes.shape[-1], dtype=torch.float64, device="cuda")
    out[..., 0::2] = table[(codes % 16).long()]
    out[..., 1::2] = table[(codes // 16).long()]
    return out


def exact(case, seed):
    """The operators' definitions in 64 bits; a plan has whole numbers only."""
    op = case["op"]
    if op == "plan":
        return None
    s = prepare(case, seed)
    if op == "matvec":
        x, sg = _turn(s["x"].double(), s["group"]), s["sg"].double()
        y = torch.zeros(s["tokens"], s["N"], dtype=torch.float64, device="cuda")
        for lo in range(0, s["N"], 2048):
            w = _values(s["qw"][lo:lo + 2048])
            w *= sg[lo:lo + 2048].repeat_interleave(s["scale_group"], 1)
            y[:, lo:lo + 2048] = torch.einsum("mk,nk->mn", x, w)
        return y if s["b"] is None else y + s["b"].double()
    if op == "append":
        def there_and_back(x):
            out = torch.empty(x.shape, dtype=torch.float64, device="cuda")
            for lo in range(0, x.shape[0], 2048):
                y = _turn(x[lo:lo + 2048].double(), s["group"])
                scale = (y.abs().amax(-1, keepdim=True) / 7).to(torch.bfloat16).double()
                r = y / torch.where(scale > 0, scale, 1.0)
                c = torch.where(r >= 0, (r + 0.5).floor(), (r - 0.5).ceil()).clamp(-7, 7)
                out[lo:lo + 2048] = _turn(c * scale, s["group"])
            return out
        return there_and_back(s["k"]), there_and_back(s["v"])
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    kc, ks, vc, vs = s["cache"]
    cu, lens, G = s["cu_q"].tolist(), s["lens"].tolist(), s["heads"] // s["kv_heads"]
    for b in range(s["requests"]):
        n, a, z = lens[b], cu[b], cu[b + 1]
        at = s["table"][b, :-(-n // s["page"])].long()
        hidden = torch.arange(n, device="cuda") > (n - (z - a) + torch.arange(z - a, device="cuda"))[:, None]
        for h in range(s["kv_heads"]):
            k, v = (_turn(_values(c[at, h].flatten(0, 1)[:n]) * w[at, h].flatten()[:n].double()[:, None], s["group"])
                    for c, w in ((kc, ks), (vc, vs)))
            q = s["q"][a:z, h * G:(h + 1) * G].double()
            p = torch.einsum("tgd,ld->gtl", q, k) * s["scale"]
            p = torch.softmax(p.masked_fill(hidden, float("-inf")), -1).nan_to_num(0.0)
            out[a:z, h * G:(h + 1) * G] = torch.einsum("gtl,ld->tgd", p, v)
    return out

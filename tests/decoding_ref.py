"""Plain 64-bit restatements of the decoding operators (group-scaled linear,
INT4 cache, attention over it, plan of a step), for the tests.  torch on the
CPU and Python loops; nothing of the package."""
import numpy as np
import torch


def hadamard(n: int) -> torch.Tensor:
    """H_n by the digit rule: (-1)^(base-4 digits that agree) / sqrt(n)."""
    i = np.arange(n)
    agree = np.zeros((n, n), dtype=int)
    d = 1
    while d < n:
        agree += ((i // d) % 4)[:, None] == ((i // d) % 4)[None, :]
        d *= 4
    return torch.from_numpy((-1.0) ** agree / np.sqrt(n))


def rotate(x: torch.Tensor, group: int) -> torch.Tensor:
    """x [..., K] float64 times I (x) H_group (group 0: unchanged)."""
    if not group:
        return x
    return (x.reshape(*x.shape[:-1], -1, group) @ hadamard(group)).reshape(x.shape)


def unpack(q: torch.Tensor) -> torch.Tensor:
    """uint8 [..., n] -> int64 [..., 2 n]."""
    q = q.to(torch.int64)
    both = torch.stack([q & 15, q >> 4], -1).reshape(*q.shape[:-1], -1)
    return torch.where(both > 7, both - 16, both)


def quantize_blocks(y: torch.Tensor, block: int):
    """fp32 [..., K] -> (int64 codes [..., K], bf16 scales [..., K / block]):
    the definition in fp32, one operation at a time."""
    y = y.reshape(*y.shape[:-1], -1, block).float()
    s = (y.abs().amax(-1) / torch.tensor(7.0)).to(torch.bfloat16)
    s = torch.where(s.float() < 2.0 ** -100, torch.zeros_like(s), s)
    inv = torch.where(s == 0, torch.zeros(()), torch.tensor(1.0) / s.float())
    v = y * inv[..., None]
    # |v| < 7.04: v + 0.5 is exact in 64 bits, so this is half away from zero
    c = (torch.sign(v.double()) * torch.floor(v.double().abs() + 0.5)).clamp(-7, 7)
    return c.reshape(*c.shape[:-2], -1).to(torch.int64), s


def linear(xr, qw, sg, bias):
    """(exact product, sum of |terms|) in float64."""
    K = xr.shape[1]
    w = unpack(qw).double() * sg.double().repeat_interleave(K // sg.shape[1], 1)
    t = xr.double() @ w.T
    return (t if bias is None else t + bias.double()), xr.double().abs() @ w.abs().T


def cache_rows(codes, scales, table, n, h):
    """Rotated float64 rows [n, D] of one request and head."""
    page = codes.shape[2]
    ids = table[:-(-n // page)].long()
    c = unpack(codes[ids, h].reshape(-1, codes.shape[3])[:n]).double()
    return c * scales[ids, h].reshape(-1)[:n].double()[:, None]


def ks_rows(scales, table, n, h):
    page = scales.shape[2]
    return scales[table[:-(-n // page)].long(), h].reshape(-1)[:n].double()


def attention(q, cache, table, lens, cu_q, scale, group, dead=()):
    """(out, tolerance norm, terms) float64: out [T, heads, D]; per row an
    allowance for the kernel's roundings as derived in test_gpu_kv4.py.
    dead: (request, table entry) pairs whose keys are taken as hidden."""
    kc, ks, vc, vs = cache
    T, Hq, D = q.shape
    Hkv, page = kc.shape[1], kc.shape[2]
    G = Hq // Hkv
    out = torch.zeros(T, Hq, D, dtype=torch.float64)
    allow = torch.zeros(T, Hq, dtype=torch.float64)
    for b in range(len(lens)):
        n, a, z = int(lens[b]), int(cu_q[b]), int(cu_q[b + 1])
        if n == 0:
            continue
        hidden_page = torch.zeros(n, dtype=torch.bool)
        row = table[b].clone()
        for (rb, j) in dead:
            if rb == b:
                hidden_page[j * page:(j + 1) * page] = True
                row[j] = 0
        for h in range(Hkv):
            k = cache_rows(kc, ks, row, n, h)
            v = cache_rows(vc, vs, row, n, h)
            for i in range(z - a):
                seen = (torch.arange(n) <= n - (z - a) + i) & ~hidden_page
                if not seen.any():
                    continue
                kk, vv = k[seen], v[seen]
                for hq in range(h * G, (h + 1) * G):
                    qr = rotate(q[a + i, hq].double(), group)
                    s = kk @ qr * scale
                    p = torch.softmax(s, 0)
                    out[a + i, hq] = rotate(p @ vv, group)
                    # scores: 16-bit queries (half a step of the row's largest
                    # / 32000: 2^-16 of it), fp32 rotation (1e-5 of it), exact
                    # sums, three fp32 products (2^-17 of the terms)
                    l1 = kk.abs() @ (qr.abs() * 2.0 ** -17 + qr.abs().max() * (2.0 ** -16 + 1e-5)) * abs(scale)
                    # and the maximum taken off in fp32 (2^-24 of the score), exp2f 2 ulp
                    ds = float((l1 + s.abs() * 2.0 ** -22).max()) + 2.0 ** -22
                    # weights: both the numerator and the sum move by ds; P s_v in
                    # f16 (2^-11); fp32 sums 2^-16
                    e = float(np.expm1(2 * ds)) + 2.0 ** -11 + 2.0 ** -16
                    allow[a + i, hq] = e * (p @ vv.abs()).norm() + 2.0 ** -8 * out[a + i, hq].norm()
                    # the offset of the values' codes comes and goes in every
                    # tile: 8 sum p s_v, off by an ulp (2^-23) in each of five
                    # steps, and weights below the f16 range (half a step,
                    # 2^-25 of a unit that is 2^-6 of the reference, times
                    # twice the largest scale), in each of D values
                    sv = ks_rows(vs, row, n, h)[seen]
                    allow[a + i, hq] += D ** 0.5 * (8 * 5 * 2.0 ** -23 * float(p @ sv) + 7 * 2.0 ** -30 * float(sv.max()) * len(sv))
    return out, allow


def plan(cached, new, table, free, count, page, max_tokens):
    """The step's bookkeeping with Python lists.  table and free are changed."""
    B, most, cap = len(cached), len(table[0]) if table else 0, len(free)
    bad = dict(seq_lens=list(cached), cu_q=[0] * (B + 1), slots=[-1] * max_tokens,
               positions=[-1] * max_tokens, result=[count, 0, 0, 0])

    def refuse(why):
        bad["result"][3] = why
        return bad
    pages = lambda n: -(-n // page)   # noqa: E731
    why = 0
    for c, n in zip(cached, new):
        if c < 0 or pages(c) > most:
            why = max(why, 4)
        elif n >= 0 and (pages(c + n) > most or c + n > 2 ** 31 - 1):
            why = max(why, 2)
    if why:
        return refuse(why)
    back = [i for c, n, row in zip(cached, new, table) if n < 0 for i in row[:pages(c)]]
    if count < 0 or count + len(back) > cap:
        return refuse(4)
    if sum(n for n in new if n > 0) > max_tokens:
        return refuse(3)
    need = sum(pages(c + n) - pages(c) for c, n in zip(cached, new) if n >= 0)
    if need > count + len(back):
        return refuse(1)
    stack = list(free[:count]) + back
    free[count:count + len(back)] = back
    lens, cu, slots, positions = [], [0], [], []
    for b, (c, n) in enumerate(zip(cached, new)):
        if n < 0:
            lens.append(0)
            cu.append(cu[-1])
            continue
        for j in range(pages(c), pages(c + n)):
            table[b][j] = stack.pop()
        for pos in range(c, c + n):
            slots.append(table[b][pos // page] * page + pos % page)
            positions.append(pos)
        lens.append(c + n)
        cu.append(cu[-1] + n)
    tail = [-1] * (max_tokens - len(slots))
    return dict(seq_lens=lens, cu_q=cu, slots=slots + tail, positions=positions + tail,
                result=[len(stack), need, cu[-1], 0])

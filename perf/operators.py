"""The operators of the softmax-attention layers that stand between delta-rule layers in a hybrid
stack, as measured cases: pages of a key-value cache given to requests, the norm and rotation of
queries and keys (forward, backward, and the form that fills the cache), and the attention of one
new token over that cache.

``listed()`` and ``draw()`` give cases, ``prepare()`` what a program has in hand before the call,
``run()`` one pass: in plain torch operations where ``own`` is false, through
``gated_delta_rule_107_b200.binding`` where it is true.  ``exact()`` evaluates the definitions in
64 bits.  Lengths depend on the case alone, values and page numbers on the seed.
"""
import math
import random

import torch

own = False

EPS = 1e-6  # of the norm
DTYPE = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------------------------ cases
def listed():
    return [
        # a decoding step of 61 running requests and 3 empty places: one new token each
        dict(name="pages_decode_64", op="pages", requests=64, new="one", longest=8192, page=16),
        # admission of 509 requests at once, prompts of up to 4096 tokens, some with a cached prefix
        dict(name="pages_prefill_509", op="pages", requests=509, new="ragged", longest=4096, page=64),
        # training forward at the headline workload's tokens (8 x 4096), 8 query and 2 key heads
        dict(name="qkrope_fwd_8x4096_bf16", op="fwd", B=8, T=4096, Hq=8, Hk=2, d=128, rot=128, interleaved=False,
             dtype="bf16", theta=10000.0, far=0),
        # a small fp32 layer (64 channels, half of them rotated, neighbouring pairs) on a ragged length
        dict(name="qkrope_fwd_3x777_f32", op="fwd", B=3, T=777, Hq=6, Hk=3, d=64, rot=32, interleaved=True,
             dtype="f32", theta=10000.0, far=0),
        # training backward at the headline workload's tokens
        dict(name="qkrope_bwd_8x4096_bf16", op="bwd", B=8, T=4096, Hq=8, Hk=2, d=128, rot=128, interleaved=False,
             dtype="bf16", theta=10000.0, far=0),
        # training backward of one long sequence (32768 tokens, 16 query heads), positions far out
        dict(name="qkrope_bwd_1x32768_bf16", op="bwd", B=1, T=32768, Hq=16, Hk=4, d=128, rot=64, interleaved=False,
             dtype="bf16", theta=1000000.0, far=900000),
        # a decoding step of 64 requests: rotate, and put the new keys and values into their pages
        dict(name="qkrope_cache_64", op="cache", N=64, padded=3, Hq=16, Hk=2, d=128, rot=128, interleaved=False,
             dtype="bf16", theta=1000000.0, page=16),
        # prompts of 8191 tokens together, padded by one
        dict(name="qkrope_cache_8192", op="cache", N=8192, padded=1, Hq=16, Hk=2, d=128, rot=128, interleaved=False,
             dtype="bf16", theta=1000000.0, page=64),
        # one user's chat: a single request of 2000 tokens (latency)
        dict(name="attn_1x2000_bf16", op="attn", requests=1, longest=2000, ragged=False, Hq=8, Hk=2, d=128, window=0,
             dtype="bf16", page=16),
        # a serving batch: 64 requests of 1 to 16384 tokens, two of the places empty
        dict(name="attn_64x16384_bf16", op="attn", requests=64, longest=16384, ragged=True, Hq=16, Hk=2, d=128,
             window=0, dtype="bf16", page=16),
        # three long documents
        dict(name="attn_3x200001_bf16", op="attn", requests=3, longest=200001, ragged=False, Hq=16, Hk=4, d=128,
             window=0, dtype="bf16", page=64),
        # a small fp32 layer with a sliding window, a key head for every query head, pages of 7 tokens
        dict(name="attn_17x5000_f32", op="attn", requests=17, longest=5000, ragged=True, Hq=6, Hk=6, d=64, window=1000,
             dtype="f32", page=7),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["pages", "fwd", "bwd", "cache", "attn", "attn"])
    page = rng.choice([1, 7, 16, 32, 64, 128])
    if op == "pages":
        new = rng.choice(["one", "ragged"])
        return dict(op=op, requests=_log_int(rng, 1, 500), new=new, longest=_log_int(rng, 16, 4000),
                    page=max(page, 7))
    d = rng.choice([64, 128])
    Hk = rng.choice([1, 2, 3, 4, 8])
    Hq = Hk * rng.choice([1, 2, 3, 4, 5, 8])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    size = 2 if dtype == "bf16" else 4
    if op == "attn":
        requests = _log_int(rng, 1, 200)
        most = 8.0e8 / (requests * Hk * d * 2 * size)  # bytes of the cache, ragged or not
        longest = _log_int(rng, 1, max(1, min(200000, int(most))))
        return dict(op=op, requests=requests, longest=longest, ragged=rng.random() < 0.6, Hq=Hq, Hk=Hk, d=d,
                    window=rng.choice([0, 0, 0, _log_int(rng, 1, 8192)]), dtype=dtype, page=page)
    rot = rng.choice([d, d, d // 2, d // 4])
    style = dict(Hq=Hq, Hk=Hk, d=d, rot=rot, interleaved=rng.random() < 0.3, dtype=dtype,
                 theta=rng.choice([10000.0, 1000000.0]))
    most = int(1.0e8 / ((Hq + Hk) * d * size))  # bytes of the tokens' queries and keys
    if op == "cache":
        N = _log_int(rng, 1, min(16384, most))
        return dict(op=op, N=N, padded=rng.choice([0, N // 9]), page=page, **style)
    B = rng.choice([1, 2, 3, 8])
    return dict(op=op, B=B, T=_log_int(rng, 1, max(1, min(32768, most // B))), far=rng.choice([0, 0, 1000000]), **style)


# ------------------------------------------------------------------------------------ inputs
def _lengths(case):
    """Host lists of the case's lengths: (cached, new) for pages, the cached lengths for attn."""
    r = random.Random("%s %s %s %s" % (case["op"], case["requests"], case["longest"], case["page"]))
    R, most = case["requests"], case["longest"]
    if case["op"] == "pages":
        if case["new"] == "one":
            cached = [r.randint(1, most) for _ in range(R)]
            new = [1] * R
            if R >= 16:  # places without a request
                for i in (3, R // 2, R - 1):
                    cached[i] = new[i] = 0
        else:
            cached = [r.choice([0, 0, 0, r.randint(0, 512)]) for _ in range(R)]
            new = [r.randint(1, most) for _ in range(R)]
            if R >= 16:
                new[5] = 0
        return cached, new
    if not case["ragged"]:
        return [most] * R
    lens = [_log_int(r, 1, most) if r.random() < 0.3 else r.randint(max(1, most // 4), most) for _ in range(R)]
    lens[0] = most
    if R >= 16:
        lens[R // 3] = lens[R - 1] = 0
    return lens


def _ceil(a, b):
    return -(-a // b)


def _inv_freq(case, dev):
    i = torch.arange(0, case["rot"], 2, dtype=torch.float64, device=dev)
    return case["theta"] ** (-i / case["rot"])


def prepare(case, seed):
    dev = torch.device("cuda", torch.cuda.current_device())
    g = torch.Generator(device=dev).manual_seed(seed)

    def randn(*shape, dtype=torch.float32, scale=1.0):
        return (torch.randn(*shape, device=dev, generator=g) * scale).to(dtype)

    def ints(v, dtype=torch.int32):
        return torch.tensor(v, dtype=dtype, device=dev)

    s = dict(case)
    if case["op"] == "pages":
        cached, new = _lengths(case)
        ps, R = case["page"], case["requests"]
        have = [_ceil(c, ps) for c in cached]
        width = max(_ceil(c + n, ps) for c, n in zip(cached, new)) + 2
        need = sum(_ceil(c + n, ps) for c, n in zip(cached, new))
        pages = torch.randperm(need + R + 8, device=dev, generator=g).to(torch.int32)
        table = torch.full((R, width), -1, dtype=torch.int32, device=dev)
        mask = torch.arange(width, device=dev)[None, :] < ints(have, torch.int64)[:, None]
        table[mask] = pages[:sum(have)]
        s.update(cached=ints(cached), new=ints(new), table=table, free_pages=pages[sum(have):].contiguous(),
                 n_free=ints([pages.numel() - sum(have)]), tokens=sum(new) + 5)  # a padded batch of tokens
        return s
    dt = DTYPE[case["dtype"]]
    d, Hq, Hk = case["d"], case["Hq"], case["Hk"]
    if case["op"] == "attn":
        lens, ps = _lengths(case), case["page"]
        R, width = len(lens), max(1, _ceil(max(lens), ps))
        used = [_ceil(n, ps) for n in lens]
        P = sum(used) + 1
        table = torch.full((R, width), -1, dtype=torch.int32, device=dev)
        mask = torch.arange(width, device=dev)[None, :] < ints(used, torch.int64)[:, None]
        table[mask] = (torch.randperm(P - 1, device=dev, generator=g) + 1).to(torch.int32)  # page 0 is nobody's
        s.update(q=randn(R, Hq, d, dtype=dt, scale=1.5), k_cache=randn(P, ps, Hk, d, dtype=dt),
                 v_cache=randn(P, ps, Hk, d, dtype=dt), table=table, lens=ints(lens), most=max(lens))
        return s
    w = dict(wq=1.0 + randn(d, scale=0.2), wk=1.0 + randn(d, scale=0.2), inv_freq=_inv_freq(case, dev))
    if case["op"] == "cache":
        N, ps = case["N"], case["page"]
        qkv = randn(N, (Hq + 2 * Hk) * d, dtype=dt, scale=2.0)  # one fused projection, as a layer has it
        q, k, v = (x.unflatten(-1, (-1, d)) for x in qkv.split([Hq * d, Hk * d, Hk * d], -1))
        live = N - case["padded"]
        P = _ceil(N, ps) + 9
        slots = torch.randperm((P - 1) * ps, device=dev, generator=g)[:N] + ps  # page 0 is nobody's
        if N > 256:  # prompts: runs of neighbouring slots
            slots = (torch.randperm(P - 1, device=dev, generator=g)[:_ceil(N, ps), None] * ps + ps
                     + torch.arange(ps, device=dev)).reshape(-1)[:N].contiguous()
        slots[live:] = -1
        s.update(q=q, k=k, v=v, slots=slots, positions=torch.randint(0, 131072, (N,), device=dev, generator=g,
                                                                     dtype=torch.int32),
                 k_cache=randn(P, ps, Hk, d, dtype=dt), v_cache=randn(P, ps, Hk, d, dtype=dt), **w)
        return s
    B, T = case["B"], case["T"]
    qkv = randn(B, T, (Hq + 2 * Hk) * d, dtype=dt, scale=2.0)
    q, k, _ = (x.unflatten(-1, (-1, d)) for x in qkv.split([Hq * d, Hk * d, Hk * d], -1))
    s.update(q=q, k=k, positions=(torch.arange(T, device=dev, dtype=torch.int32) + case["far"]).expand(B, T).contiguous(),
             **w)
    if case["op"] == "bwd":
        s.update(dq_out=randn(B, T, Hq, d, dtype=dt), dk_out=randn(B, T, Hk, d, dtype=dt))
    return s


# ------------------------------------------------------------------------------------ plain forms
def _cos_sin(positions, inv_freq):
    a = positions.double()[..., None] * inv_freq  # far positions: the angle in 64 bits
    return a.cos().float()[..., None, :], a.sin().float()[..., None, :]


def _pairs(x, rot, interleaved):
    r = x[..., :rot]
    return (r[..., 0::2], r[..., 1::2]) if interleaved else (r[..., : rot // 2], r[..., rot // 2:])


def _join(a, b, rest, interleaved):
    r = torch.stack((a, b), -1).flatten(-2) if interleaved else torch.cat((a, b), -1)
    return torch.cat((r, rest), -1)


def _plain_norm_rotate(x, w, cos, sin, rot, interleaved):
    f = x.float()
    y = f * torch.rsqrt((f * f).mean(-1, keepdim=True) + EPS) * w
    a, b = _pairs(y, rot, interleaved)
    return _join(a * cos - b * sin, b * cos + a * sin, y[..., rot:], interleaved).to(x.dtype)


def _plain_norm_rotate_bwd(x, w, dy, cos, sin, rot, interleaved):
    f, gy = x.float(), dy.float()
    a, b = _pairs(gy, rot, interleaved)
    gr = _join(a * cos + b * sin, b * cos - a * sin, gy[..., rot:], interleaved)  # the rotation back
    r = torch.rsqrt((f * f).mean(-1, keepdim=True) + EPS)
    n = f * r
    gn = gr * w
    dx = r * (gn - n * (gn * n).mean(-1, keepdim=True))
    return dx.to(x.dtype), (gr * n).flatten(0, -2).sum(0)


def _plain_pages(s):
    ps, table = s["page"], s["table"]
    cached, new = s["cached"].long(), s["new"].long()
    lens = cached + new
    have, need = (cached + ps - 1) // ps, (lens + ps - 1) // ps
    zero = torch.zeros(1, dtype=torch.int64, device=table.device)
    cu_new = torch.cat((zero, new.cumsum(0)))
    taken = torch.cat((zero, (need - have).cumsum(0)))
    n_free = s["n_free"].long()
    col = torch.arange(table.shape[1], device=table.device)[None, :]
    nth = taken[:-1, None] + col - have[:, None]  # the nth page that is taken, from the stack's top
    page = s["free_pages"][(n_free - 1 - nth).clamp(0, s["free_pages"].numel() - 1)]
    page = torch.where(nth < n_free, page, torch.full_like(page, -1))
    table = torch.where((col >= have[:, None]) & (col < need[:, None]), page, table)
    t = torch.arange(s["tokens"], device=table.device)
    r = (torch.searchsorted(cu_new, t, right=True) - 1).clamp(max=cached.numel() - 1)
    live = t < cu_new[-1]
    pos = torch.where(live, t - cu_new[r] + cached[r], torch.zeros_like(t))
    at = table[r, (pos // ps).clamp(max=table.shape[1] - 1)].long()
    slots = torch.where(live & (at >= 0), at * ps + pos % ps, torch.full_like(t, -1))
    return (lens.int(), cu_new.int(), pos.int(), slots, (n_free - taken[-1]).int(), table)


def _plain_attn(s):
    q, ps = s["q"], s["page"]
    R, Hq, d = q.shape
    Hk = s["k_cache"].shape[2]
    t = torch.arange(s["most"], device=q.device)
    lens = s["lens"].long()[:, None]
    seen = t[None, :] < lens
    if s["window"]:
        seen = seen & (t[None, :] >= lens - s["window"])
    at = s["table"].long()[:, t // ps].clamp(min=0) * ps + t % ps  # [R, L]
    k = s["k_cache"].flatten(0, 1)[at].float().permute(0, 2, 3, 1)  # [R, Hk, d, L]
    v = s["v_cache"].flatten(0, 1)[at].float().transpose(1, 2)  # [R, Hk, L, d]
    x = torch.matmul(q.float().view(R, Hk, Hq // Hk, d), k) * (1.0 / math.sqrt(d))
    x = x.masked_fill(~seen[:, None, None, :], -math.inf)
    m = x.amax(-1, keepdim=True).clamp(min=torch.finfo(torch.float32).min)  # rows that see nothing
    p = torch.exp(x - m)
    z = p.sum(-1, keepdim=True)
    o = torch.matmul(p, v) / torch.where(z > 0, z, torch.ones_like(z))
    lse = torch.where(z > 0, m + z.log(), torch.full_like(z, -math.inf))
    return o.view(R, Hq, d).to(q.dtype), lse.view(R, Hq)


def _plain(s):
    op = s["op"]
    if op == "pages":
        return _plain_pages(s)
    if op == "attn":
        return _plain_attn(s)
    cos, sin = _cos_sin(s["positions"], s["inv_freq"])
    style = (cos, sin, s["rot"], s["interleaved"])
    if op == "bwd":
        dq, dwq = _plain_norm_rotate_bwd(s["q"], s["wq"], s["dq_out"], *style)
        dk, dwk = _plain_norm_rotate_bwd(s["k"], s["wk"], s["dk_out"], *style)
        return dq, dk, dwq, dwk
    q, k = _plain_norm_rotate(s["q"], s["wq"], *style), _plain_norm_rotate(s["k"], s["wk"], *style)
    if op == "fwd":
        return q, k
    skip = (s["slots"] < 0)[:, None, None]  # padding: written back what the nobody's row holds
    at = s["slots"].clamp(min=0)
    for_k, for_v = s["k_cache"].flatten(0, 1), s["v_cache"].flatten(0, 1)
    for_k[at] = torch.where(skip, for_k[0], k)
    for_v[at] = torch.where(skip, for_v[0], s["v"])
    return q, s["k_cache"], s["v_cache"]


def run(s):
    if not own:
        return _plain(s)
    from gated_delta_rule_107_b200 import binding
    op = s["op"]
    if op == "attn":
        return binding.delta_rule_attn_decode(s["q"], s["k_cache"], s["v_cache"], s["table"], s["lens"],
                                              window=s["window"], want_lse=True)
    if op == "cache":
        q = binding.delta_rule_qkrope_cache(s["q"], s["k"], s["v"], s["wq"], s["wk"], s["inv_freq"], s["positions"],
                                            s["slots"], s["k_cache"], s["v_cache"], interleaved=s["interleaved"])
        return q, s["k_cache"], s["v_cache"]
    if op == "fwd":
        return binding.delta_rule_qkrope(s["q"], s["k"], s["wq"], s["wk"], s["inv_freq"], s["positions"],
                                         interleaved=s["interleaved"])
    if op == "bwd":
        return binding.delta_rule_qkrope_bwd(s["q"], s["k"], s["wq"], s["wk"], s["inv_freq"], s["dq_out"], s["dk_out"],
                                             s["positions"], interleaved=s["interleaved"])
    return binding.delta_rule_pages(s["cached"], s["new"], s["free_pages"], s["n_free"], s["table"], s["page"],
                                    s["tokens"]) + (s["table"],)


# ------------------------------------------------------------------------------------ work
def work(case):
    if case["op"] == "pages":
        cached, new = _lengths(case)
        ps, R, N = case["page"], case["requests"], sum(new) + 5
        first = sum(c // ps < _ceil(c, ps) and n > 0 for c, n in zip(cached, new))  # last page of the prefix
        taken = sum(_ceil(c + n, ps) - _ceil(c, ps) for c, n in zip(cached, new))
        return {"bytes": 8 * R + 4 + 4 * first + 4 * taken + 4 * taken + 4 * R + 4 * (R + 1) + 4 + 12 * N,
                "flops": 4 * N}
    e, d, Hq, Hk = (2 if case["dtype"] == "bf16" else 4), case["d"], case["Hq"], case["Hk"]
    if case["op"] == "attn":
        lens = _lengths(case)
        seen = sum(min(n, case["window"]) if case["window"] else n for n in lens)
        pages = sum(_ceil(n, case["page"]) - (max(0, n - case["window"]) // case["page"] if case["window"] else 0)
                    for n in lens)
        R = len(lens)
        return {"bytes": 2 * seen * Hk * d * e + 2 * R * Hq * d * e + 4 * R * Hq + 4 * R + 4 * pages,
                "flops": 4 * seen * Hq * d}
    small = 2 * 4 * d + 8 * (case["rot"] // 2)
    if case["op"] == "cache":
        N, live = case["N"], case["N"] - case["padded"]
        return {"bytes": (2 * N * Hq + 4 * live * Hk) * d * e + 12 * N + small, "flops": 8 * N * (Hq + Hk) * d}
    N = case["B"] * case["T"]
    if case["op"] == "fwd":
        return {"bytes": 2 * N * (Hq + Hk) * d * e + 4 * N + small, "flops": 8 * N * (Hq + Hk) * d}
    return {"bytes": 3 * N * (Hq + Hk) * d * e + 4 * N + small + 2 * 4 * d, "flops": 16 * N * (Hq + Hk) * d}


# ------------------------------------------------------------------------------------ 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "pages":
        return _exact_pages(case, s)
    if case["op"] == "attn":
        return _exact_attn(s)
    theta = torch.outer(s["positions"].double().flatten(), s["inv_freq"])  # [N, rot / 2]
    turn = torch.polar(torch.ones_like(theta), theta)[:, None, :]
    rot, style = case["rot"], case["interleaved"]

    def rotated(y, by):  # [N, H, d]: channel pairs as complex numbers, times e^(i theta)
        head = y[..., :rot]
        z = torch.view_as_complex((head.unflatten(-1, (-1, 2)) if style else head.unflatten(-1, (2, -1)).transpose(-1, -2)).contiguous()) * by
        out = torch.view_as_real(z)
        out = out.flatten(-2) if style else out.transpose(-1, -2).flatten(-2)
        return torch.cat((out, y[..., rot:]), -1)

    def forward(x, w):
        y = x.double().reshape(-1, *x.shape[-2:])
        y = y / ((y.square().sum(-1, keepdim=True) / y.shape[-1]) + EPS).sqrt() * w.double()
        return rotated(y, turn)

    if case["op"] == "bwd":
        def backward(x, w, dy):
            f = x.double().reshape(-1, *x.shape[-2:])
            gr = rotated(dy.double().reshape(-1, *x.shape[-2:]), turn.conj())
            rms = ((f.square().sum(-1, keepdim=True) / f.shape[-1]) + EPS).sqrt()
            gw = gr * w.double()
            dx = gw / rms - f * ((gw * f).sum(-1, keepdim=True) / (f.shape[-1] * rms**3))
            return dx.view(x.shape), torch.einsum("nhd,nhd->d", gr, f / rms)

        dq, dwq = backward(s["q"], s["wq"], s["dq_out"])
        dk, dwk = backward(s["k"], s["wk"], s["dk_out"])
        return dq, dk, dwq, dwk
    q, k = forward(s["q"], s["wq"]), forward(s["k"], s["wk"])
    if case["op"] == "fwd":
        return q.view(s["q"].shape), k.view(s["k"].shape)
    live = s["slots"] >= 0
    caches = []
    for cache, new in ((s["k_cache"], k), (s["v_cache"], s["v"].double())):
        c = cache.double()
        c.view(-1, *c.shape[2:])[s["slots"][live]] = new[live]
        caches.append(c)
    return (q.view(s["q"].shape), *caches)


def _exact_pages(case, s):
    cached, new = s["cached"].tolist(), s["new"].tolist()
    table, stack, ps = s["table"].tolist(), s["free_pages"].tolist()[: int(s["n_free"])], case["page"]
    left, positions, slots, cu_new = len(stack), [], [], [0]
    for r, (c, n) in enumerate(zip(cached, new)):
        for j in range(_ceil(c, ps), _ceil(c + n, ps)):
            left -= 1
            table[r][j] = stack[left] if left >= 0 else -1
        for p in range(c, c + n):
            page = table[r][p // ps]
            positions.append(p)
            slots.append(page * ps + p % ps if page >= 0 else -1)
        cu_new.append(cu_new[-1] + n)
    pad = s["tokens"] - len(positions)
    dev = s["table"].device

    def t(v, dtype=torch.int32):
        return torch.tensor(v, dtype=dtype, device=dev)

    return (t([c + n for c, n in zip(cached, new)]), t(cu_new), t(positions + [0] * pad), t(slots + [-1] * pad, torch.int64),
            t([left]), t(table))


def _exact_attn(s):
    q, ps = s["q"].double(), s["page"]
    R, Hq, d = q.shape
    Hk = s["k_cache"].shape[2]
    o = torch.zeros_like(q)
    lse = torch.full((R, Hq), -math.inf, dtype=torch.float64, device=q.device)
    for r, n in enumerate(s["lens"].tolist()):
        first = max(0, n - s["window"]) if s["window"] else 0
        if n <= first:
            continue
        pages = s["table"][r, first // ps: _ceil(n, ps)].long()
        cut = slice(first % ps, first % ps + n - first)
        k, v = (c[pages].flatten(0, 1)[cut].double() for c in (s["k_cache"], s["v_cache"]))
        x = torch.einsum("hgd,thd->hgt", q[r].view(Hk, -1, d), k) / math.sqrt(d)
        lse[r] = torch.logsumexp(x, -1).flatten()
        o[r] = torch.einsum("hgt,thd->hgd", torch.softmax(x, -1), v).reshape(Hq, d)
    return o, lse

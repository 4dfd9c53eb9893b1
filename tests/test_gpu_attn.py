"""The operators of a softmax-attention layer beside the delta rule against the fp64 reference in
oracle/attn.py: cache pages, norm with rotation (forward, backward, into the cache), attention of
one new token over the paged cache, and a run of them together.

Tolerances, per element, from the arithmetic.  A rounding to type t is off by at most
finfo(t).eps / 2 of the value.  fp32 steps are counted in units of 2^-24 of the largest operand:
  norm and rotation: y takes a sum of d squares by pairs (each term's sum at most 8 + log2(32)
    roundings deep), a root, two products and a rotation of two terms whose angle's cosine and sine
    are off by 2^-22 or less (for bf16 results 2^-20): 64 units of the row's largest |y| cover them;
    gradients the same with the row's largest |dy w| / rms, times (1 + the largest |n|^2) for the projection's term.
  attention: a score's sum of d products is off by at most (d + 4) 2^-23 sum |q_c k_c| scale; the
    weights then by twice that, relatively, and the exponential's 2^-21; splitting p into two bf16
    numbers leaves 2^-16 of it; sums over n tokens, 16 a step, four warps and up to 296 runs, (n / 16
    + 64) 2^-23 -- all relative to the largest |v|.
"""
import numpy as np
import pytest
import torch

from gated_delta_rule_107_b200 import binding
from oracle import attn as oa
from parity_util import np64

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}
HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}


def _rng(seed):
    return torch.Generator().manual_seed(seed)


def _randn(g, *shape, dtype="f32", scale=1.0):
    return (torch.randn(*shape, generator=g) * scale).to(DT[dtype]).cuda()


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _within(got, ref, tol, what):
    got = np64(got)
    assert got.shape == ref.shape, what
    bad = ~(np.abs(got - ref) <= tol)
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} off, worst {np.nanmax(np.abs(got - ref) / np.maximum(tol, 1e-300))} x tol"


# ------------------------------------------------------------------------------------ pages
def _pages_case(R, width, page, F, tokens, cached, fresh, n_free=None, seed=0):
    g = _rng(seed)
    table = torch.randint(-3, 1000, (R, width), generator=g, dtype=torch.int32).cuda()
    free = torch.randperm(F, generator=g).to(torch.int32).cuda()
    nf = _i32([F if n_free is None else n_free])
    before = table.clone()
    got = binding.delta_rule_pages(_i32(cached), _i32(fresh), free, nf, table, page, tokens)
    torch.cuda.synchronize()
    ref = oa.pages(cached, fresh, free.cpu().numpy(), int(nf), before.cpu().numpy(), page, tokens)
    for name, a, b in zip(("lens", "cu_new", "positions", "slots", "n_left", "table"), got + (table,), ref):
        b = np.atleast_1d(b)
        assert np.array_equal(a.cpu().numpy().astype(np.int64), b), name
    return got, table


@pytest.mark.parametrize("R,page,most", ((1, 16, 40), (3, 1, 9), (64, 16, 300), (257, 7, 60), (700, 64, 500), (8192, 16, 20)))
def test_pages_match_reference(R, page, most):
    rng = np.random.default_rng(R)
    cached = rng.integers(0, most, R) * (rng.random(R) < 0.7)
    fresh = rng.integers(0, most, R) * (rng.random(R) < 0.8)
    width = 2 * most // page + 2
    need = int(sum(-(-(c + f) // page) - -(-c // page) for c, f in zip(cached, fresh)))
    _pages_case(R, width, page, need + 5, int(fresh.sum()) + 3, cached.tolist(), fresh.tolist(), seed=R)


def test_pages_decoding_steps_follow_one_another():
    """Forty steps of one token: the stack's count and the table passed on, no page given twice."""
    R, page, F = 5, 4, 64
    g = _rng(1)
    table = torch.full((R, 16), -1, dtype=torch.int32, device="cuda")
    free, left = torch.randperm(F, generator=g).to(torch.int32).cuda(), _i32([F])
    lens = _i32([0, 3, 0, 7, 4])
    zero = torch.zeros_like(lens)
    lens, _, _, _, left = binding.delta_rule_pages(zero, lens, free, left, table, page, 14)
    for step in range(40):
        fresh = _i32([1, 1, 0, 1, int(step % 3 == 0)])
        cached = lens
        lens, cu, pos, slots, left = binding.delta_rule_pages(cached, fresh, free, left, table, page, R)
        n = int(cu[-1])
        rows = [r for r in range(R) if int(fresh[r])]
        assert pos[:n].tolist() == [int(cached[r]) for r in rows]
        assert slots[:n].tolist() == [int(table[r, int(cached[r]) // page]) * page + int(cached[r]) % page for r in rows]
        assert (slots[n:] == -1).all()
    used = table[table >= 0].tolist()
    assert len(used) == len(set(used)) == F - int(left)


def test_pages_edges():
    _pages_case(0, 3, 4, 5, 6, [], [])                                        # no request
    _pages_case(3, 2, 4, 9, 0, [1, 2, 3], [5, 6, 0])                          # no room for tokens
    _pages_case(3, 4, 4, 9, 5, [1, 2, 3], [5, 6, 0])                          # room for fewer tokens
    _pages_case(3, 2, 4, 9, 40, [7, 0, 30], [9, 12, 8])                       # tokens behind the table
    _pages_case(3, 8, 4, 2, 40, [7, 0, 30], [9, 12, 8])                       # a short stack
    _pages_case(3, 8, 4, 9, 40, [7, 0, 30], [9, 12, 8], n_free=0)             # an empty one
    _pages_case(3, 8, 4, 9, 40, [7, 0, 30], [9, 12, 8], n_free=100)           # counts out of range
    _pages_case(3, 8, 4, 9, 40, [7, 0, 30], [9, 12, 8], n_free=-4)
    _pages_case(2, 0, 4, 9, 6, [0, 1], [2, 2])                                # no table
    _pages_case(3, 8, 4, 9, 30, [-7, 2, 3], [9, -12, 8])                      # negative lengths
    _pages_case(2, 5, 1 << 30, 9, 7, [0, 2], [3, 4])                          # one page for everything


def test_pages_lengths_near_the_top_of_int32():
    big = 2 ** 31 - 1
    table = torch.full((2, 3), 8, dtype=torch.int32, device="cuda")
    lens, cu, pos, slots, left = binding.delta_rule_pages(_i32([big - 2, 0]), _i32([5, big]), _i32([1, 2, 3, 4]),
                                                          _i32([4]), table, 16, 8)
    torch.cuda.synchronize()
    assert lens.tolist() == [big, big] and cu.tolist() == [0, 5, big]
    assert slots[:5].tolist() == [-1] * 5                      # behind the table
    assert slots[5:].tolist() == [64, 65, 66] and left.tolist() == [1] and table.tolist() == [[8] * 3, [4, 3, 2]]


# ------------------------------------------------------------------------------------ norm and rotation
def _freq(rot, theta=10000.0):
    return theta ** (-torch.arange(0, rot, 2, dtype=torch.float64) / max(rot, 1)).cuda() if rot else None


def _qk_case(dtype, B, T, Hq, Hk, d, rot, seed, far=0, weights=True):
    g = _rng(seed)
    qkv = _randn(g, B, T, (Hq + 2 * Hk) * d, dtype=dtype, scale=2.0)
    q, k, v = (x.unflatten(-1, (-1, d)) for x in qkv.split([Hq * d, Hk * d, Hk * d], -1))
    w = [1 + _randn(g, d, scale=0.3) if weights else None for _ in range(2)]
    pos = (torch.randint(0, 5000, (B, T), generator=g) + far).to(torch.int32).cuda()
    return q, k, v, w, _freq(rot), pos


def _flat(t):
    return np64(t).reshape(-1, *t.shape[-2:])


def _check_norm(got, x, w, pos, f, interleaved, dtype, what):
    ref = oa.qkrope(_flat(x), np64(w), pos.flatten().cpu().numpy(), np.zeros(0) if f is None else np64(f), interleaved)
    tol = HALF[dtype] * np.abs(ref) + 64 * 2.0 ** -24 * np.abs(ref).max(-1, keepdims=True) * 1.5
    _within(got.reshape(-1, *got.shape[-2:]), ref, tol, what)


def _check_norm_bwd(gx, gw, x, w, pos, f, dy, interleaved, dtype, what):
    xn, wn, dyn = _flat(x), np64(w), _flat(dy)
    fn = np.zeros(0) if f is None else np64(f)
    dx, dw = oa.qkrope_bwd(xn, wn, pos.flatten().cpu().numpy(), fn, dyn, interleaved)
    rms = np.sqrt((xn * xn).mean(-1, keepdims=True) + 1e-6)
    n = xn / rms
    size = 1.5 * np.abs(dyn).max(-1, keepdims=True) * (1 if wn is None else np.abs(wn).max()) / rms
    _within(gx.reshape(dx.shape), dx, HALF[dtype] * np.abs(dx) + 64 * 2.0 ** -24 * size * (1 + (n * n).max(-1, keepdims=True)), what)
    # dw: every term is off by 64 units at most; the sum's depth is at most the terms of a lane and 64 joins
    terms = 1.5 * np.abs(dyn).max(-1, keepdims=True) * np.abs(n)
    _within(gw, dw, (64 + 64 + xn.shape[0] * xn.shape[1] / 256) * 2.0 ** -24 * terms.sum((0, 1)) + 2.0 ** -24 * np.abs(dw), what + " dw")


@pytest.mark.parametrize("dtype", ("f32", "bf16"))
@pytest.mark.parametrize("d,rot,interleaved", ((128, 128, False), (128, 64, True), (64, 64, True), (64, 16, False),
                                               (128, 0, False), (64, 32, False), (128, 32, True)))
@pytest.mark.parametrize("B,T,Hq,Hk", ((1, 1, 1, 1), (2, 37, 5, 1), (3, 129, 4, 4)))
def test_qkrope_forward_and_backward(dtype, d, rot, interleaved, B, T, Hq, Hk):
    q, k, _, (wq, wk), f, pos = _qk_case(dtype, B, T, Hq, Hk, d, rot, seed=d + rot + T)
    qo, ko = binding.delta_rule_qkrope(q, k, wq, wk, f, pos, interleaved=interleaved)
    g = _rng(9)
    dqo, dko = _randn(g, B, T, Hq, d, dtype=dtype), _randn(g, B, T, Hk, d, dtype=dtype)
    dq, dk, dwq, dwk = binding.delta_rule_qkrope_bwd(q, k, wq, wk, f, dqo, dko, pos, interleaved=interleaved)
    torch.cuda.synchronize()
    assert qo.is_contiguous() and ko.is_contiguous()
    _check_norm(qo, q, wq, pos, f, interleaved, dtype, "q_out")
    _check_norm(ko, k, wk, pos, f, interleaved, dtype, "k_out")
    _check_norm_bwd(dq, dwq, q, wq, pos, f, dqo, interleaved, dtype, "dq")
    _check_norm_bwd(dk, dwk, k, wk, pos, f, dko, interleaved, dtype, "dk")
    again = binding.delta_rule_qkrope_bwd(q, k, wq, wk, f, dqo, dko, pos, interleaved=interleaved)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(again, (dq, dk, dwq, dwk)))  # bit for bit


def test_qkrope_many_tokens_and_defaults():
    """More tokens than one sweep of the grid, default positions and weights, no heads on one side."""
    B, T, Hq, Hk, d = 2, 9001, 2, 1, 64
    q, k, _, _, f, _ = _qk_case("bf16", B, T, Hq, Hk, d, 64, seed=5, weights=False)
    pos = torch.arange(T, dtype=torch.int32, device="cuda").expand(B, T)
    qo, ko = binding.delta_rule_qkrope(q, k, inv_freq=f)
    g = _rng(6)
    dqo, dko = _randn(g, B, T, Hq, d, dtype="bf16"), _randn(g, B, T, Hk, d, dtype="bf16")
    dq, dk, dwq, dwk = binding.delta_rule_qkrope_bwd(q, k, None, None, f, dqo, dko)
    torch.cuda.synchronize()
    _check_norm(qo, q, None, pos, f, False, "bf16", "q_out")
    _check_norm(ko, k, None, pos, f, False, "bf16", "k_out")
    _check_norm_bwd(dq, dwq, q, None, pos, f, dqo, False, "bf16", "dq")
    _check_norm_bwd(dk, dwk, k, None, pos, f, dko, False, "bf16", "dk")
    only_q, none = binding.delta_rule_qkrope(q, k[:, :, :0], inv_freq=f)
    torch.cuda.synchronize()
    assert torch.equal(only_q, qo) and none.numel() == 0
    dq2, _, dwq2, dwk2 = binding.delta_rule_qkrope_bwd(q, k[:, :, :0], None, None, f, dqo, dko[:, :, :0].contiguous())
    torch.cuda.synchronize()
    assert torch.equal(dq2, dq) and (dwk2 == 0).all()
    _check_norm_bwd(dq2, dwq2, q, None, pos, f, dqo, False, "bf16", "dq alone")


def test_qkrope_single_tokens_and_one_sided_calls():
    """A decoding batch [B, 1, heads, d] sliced from its projections, and calls with queries or keys alone."""
    q, k, v, (wq, wk), f, pos = _qk_case("bf16", 9, 1, 6, 2, 128, 128, seed=17)
    assert not q.is_contiguous()
    qo, ko = binding.delta_rule_qkrope(q, k, wq, wk, f, pos)
    torch.cuda.synchronize()
    _check_norm(qo, q, wq, pos, f, False, "bf16", "q_out")
    _check_norm(ko, k, wk, pos, f, False, "bf16", "k_out")
    none, ko2 = binding.delta_rule_qkrope(q[:, :, :0], k, wq, wk, f, pos)
    q2, k2 = q[:, 0], k[:, 0]  # [N, heads, d]
    qo3, ko3 = binding.delta_rule_qkrope(q2, k2, wq, wk, f, pos.flatten())
    kc, vc = (torch.zeros(3, 4, 2, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    out = binding.delta_rule_qkrope_cache(q2[:, :0], k2, v[:, 0], wq, wk, f, pos.flatten(), torch.arange(9, device="cuda"), kc, vc)
    torch.cuda.synchronize()
    assert none.numel() == out.numel() == 0 and torch.equal(ko2, ko)
    assert torch.equal(qo3, qo[:, 0]) and torch.equal(ko3, ko[:, 0])
    assert torch.equal(kc.view(12, 2, 128)[:9], ko[:, 0]) and torch.equal(vc.view(12, 2, 128)[:9], v[:, 0])
    e = q[:0]
    empty = binding.delta_rule_qkrope(e, k[:0], wq, wk, f, pos[:0])
    g = binding.delta_rule_qkrope_bwd(e, k[:0], wq, wk, f, empty[0], empty[1], pos[:0])
    torch.cuda.synchronize()
    assert empty[0].shape == e.shape and (g[2] == 0).all() and (g[3] == 0).all()  # sums over no rows


def test_qkrope_far_positions_keep_their_angle():
    """At positions of 10^6 and 2^31 - 1 the angles are as exact as at small ones."""
    for far in (1000000, 2 ** 31 - 6000):
        q, k, _, (wq, wk), f, pos = _qk_case("f32", 1, 40, 2, 2, 64, 64, seed=7, far=far)
        qo, ko = binding.delta_rule_qkrope(q, k, wq, wk, f, pos)
        torch.cuda.synchronize()
        _check_norm(qo, q, wq, pos, f, False, "f32", f"q_out at {far}")
    neg = -pos
    qo, _ = binding.delta_rule_qkrope(q, k, wq, wk, f, neg)
    torch.cuda.synchronize()
    _check_norm(qo, q, wq, neg, f, False, "f32", "q_out at negative positions")


def test_qkrope_gradients_go_into_slices_of_one_buffer():
    B, T, Hq, Hk, d = 2, 33, 3, 2, 128
    q, k, _, (wq, wk), f, pos = _qk_case("bf16", B, T, Hq, Hk, d, 128, seed=8)
    g = _rng(2)
    dqo, dko = _randn(g, B, T, Hq, d, dtype="bf16"), _randn(g, B, T, Hk, d, dtype="bf16")
    dq, dk, dwq, dwk = binding.delta_rule_qkrope_bwd(q, k, wq, wk, f, dqo, dko, pos)
    dqkv = torch.full((B, T, (Hq + 2 * Hk) * d), 7.0, dtype=torch.bfloat16, device="cuda")
    a, b, c = (x.unflatten(-1, (-1, d)) for x in dqkv.split([Hq * d, Hk * d, Hk * d], -1))
    got = binding.delta_rule_qkrope_bwd(q, k, wq, wk, f, dqo, dko, pos, dq=a, dk=b, want_dw=False)
    torch.cuda.synchronize()
    assert got[2] is None and torch.equal(a, dq) and torch.equal(b, dk) and (c == 7.0).all()


def test_qkrope_gradient_against_differences():
    """The GPU's own forward, differenced in fp32 at steps large enough for it."""
    B, T, Hq, Hk, d = 1, 3, 1, 1, 64
    q, k, _, (wq, wk), f, pos = _qk_case("f32", B, T, Hq, Hk, d, 32, seed=12)
    q, k = q.contiguous(), k.contiguous()
    dqo, dko = _randn(_rng(3), B, T, Hq, d), torch.zeros(B, T, Hk, d, device="cuda")
    dq, _, dwq, _ = binding.delta_rule_qkrope_bwd(q, k, wq, wk, f, dqo, dko, pos)

    def loss(x, w):
        return (binding.delta_rule_qkrope(x, k, w, wk, f, pos)[0].double() * dqo.double()).sum().item()

    h = 2.0 ** -6
    # truncation: the third derivative of a normed row's loss is below 6 |dy| sqrt(d) / rms^3 ~ 50 x h^2 / 6;
    # rounding: 192 outputs off by 2^-22 each, random in sign, over 2 h
    for t, c in ((0, 0), (0, 31), (1, 40), (2, 63), (2, 17)):
        e = torch.zeros_like(q)
        e[0, t, 0, c] = h
        fd = (loss(q + e, wq) - loss(q - e, wq)) / (2 * h)
        assert abs(fd - dq[0, t, 0, c].item()) < 50 * h * h / 6 + 192 * 2.0 ** -22 / (2 * h), (t, c)
        e = torch.zeros_like(wq)
        e[c] = h
        fd = (loss(q, wq + e) - loss(q, wq - e)) / (2 * h)
        assert abs(fd - dwq[c].item()) < 192 * 2.0 ** -22 / (2 * h) + 1e-5, c


def test_qkrope_captured_backward_beside_eager_calls():
    q, k, _, (wq, wk), f, pos = _qk_case("bf16", 2, 70, 4, 2, 128, 128, seed=13)
    g = _rng(2)
    dqo, dko = _randn(g, 2, 70, 4, 128, dtype="bf16"), _randn(g, 2, 70, 2, 128, dtype="bf16")
    eager = binding.delta_rule_qkrope_bwd(q, k, wq, wk, f, dqo, dko, pos)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = binding.delta_rule_qkrope(q, k, wq, wk, f, pos)
        grads = binding.delta_rule_qkrope_bwd(q, k, wq, wk, f, y[0], y[1], pos)
    dst = [t.clone() for t in eager]
    for _ in range(2):
        graph.replay()
    later = binding.delta_rule_qkrope_bwd(q, k, wq, wk, f, dqo, dko, pos)
    torch.cuda.synchronize()
    y2 = binding.delta_rule_qkrope(q, k, wq, wk, f, pos)
    ref = binding.delta_rule_qkrope_bwd(q, k, wq, wk, f, y2[0], y2[1], pos)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(grads, ref)) and all(torch.equal(a, b) for a, b in zip(later, dst))


# ------------------------------------------------------------------------------------ into the cache
@pytest.mark.parametrize("dtype", ("f32", "bf16"))
@pytest.mark.parametrize("N,Hq,Hk,d,page,joint", ((1, 4, 1, 128, 16, False), (7, 2, 2, 64, 7, True), (300, 16, 2, 128, 64, True),
                                                  (1000, 3, 3, 64, 1, False), (130, 2, 4, 64, 16, "heads first")))
def test_qkrope_cache(dtype, N, Hq, Hk, d, page, joint):
    q, k, v, (wq, wk), f, pos = _qk_case(dtype, 1, N, Hq, Hk, d, d // 2, seed=N)
    q, k, v, pos = q[0], k[0], v[0], pos[0].contiguous()
    P = -(-N // page) + 3
    g = _rng(N)
    both = _randn(g, P, 2, page, Hk, d, dtype=dtype)
    kc, vc = (both[:, 0], both[:, 1]) if joint is True else (both[:, 0].contiguous(), both[:, 1].contiguous())
    if joint == "heads first":
        kc, vc = (t.transpose(1, 2).contiguous().transpose(1, 2) for t in (kc, vc))
    slots = torch.randperm(P * page, generator=g)[:N]
    skip = torch.rand(N, generator=g) < 0.2
    slots[skip] = torch.tensor([-1, -7, P * page, 2 ** 40])[torch.randint(0, 4, (int(skip.sum()),), generator=g)]
    slots = slots.cuda()
    k0, v0 = kc.clone(memory_format=torch.contiguous_format), vc.clone(memory_format=torch.contiguous_format)
    qo = binding.delta_rule_qkrope_cache(q, k, v, wq, wk, f, pos, slots, kc, vc)
    torch.cuda.synchronize()
    want_q, want_k = binding.delta_rule_qkrope(q, k, wq, wk, f, pos)
    live = (slots >= 0) & (slots < P * page)
    k0.view(-1, Hk, d)[slots[live]] = want_k[live]
    v0.view(-1, Hk, d)[slots[live]] = v[live]
    torch.cuda.synchronize()
    _check_norm(want_k, k, wk, pos, f, False, dtype, "k")
    assert torch.equal(qo, want_q) and torch.equal(kc, k0) and torch.equal(vc, v0)  # the other rows untouched


# ------------------------------------------------------------------------------------ attention
def _cache(dtype, lens, page, Hk, d, seed, joint=False, extra=2, scale=1.0):
    """Pages in random order, the table's unused entries -1 and the unused rows NaN."""
    g = _rng(seed)
    used = [-(-max(n, 0) // page) for n in lens]
    P, width = sum(used) + extra, max(max(used), 1)
    both = torch.full((P, 2, page, Hk, d), float("nan"), dtype=DT[dtype], device="cuda")
    kc, vc = (both[:, 0], both[:, 1]) if joint else (both[:, 0].clone(), both[:, 1].clone())
    perm = torch.randperm(P, generator=g)
    table = torch.full((len(lens), width), -1, dtype=torch.int32)
    i = 0
    for r, n in enumerate(lens):
        for j in range(used[r]):
            table[r, j] = perm[i]
            rows = min(page, n - j * page)
            kc[perm[i], :rows] = _randn(g, rows, Hk, d, dtype=dtype, scale=scale)
            vc[perm[i], :rows] = _randn(g, rows, Hk, d, dtype=dtype)
            i += 1
    return kc, vc, table.cuda()


def _check_attn(o, lse, q, kc, vc, table, lens, dtype, scale=None, window=0, what=""):
    qn, kn, vn, tn = np64(q), np64(kc), np64(vc), table.cpu().numpy()
    ref, ref_lse = oa.attn_decode(qn, kn, vn, tn, lens, scale, window)
    R, Hq, d = q.shape
    G, page = Hq // kc.shape[2], kc.shape[1]
    sc = d ** -0.5 if scale is None else abs(scale)
    got_o, got_l = np64(o), np64(lse)
    for r in range(R):
        n = min(max(int(lens[r]), 0), tn.shape[1] * page)
        t = np.arange(max(0, n - window) if window else 0, n)
        pg = tn[r][t // page] if n else t
        t, pg = t[(pg >= 0) & (pg < kn.shape[0])], pg[(pg >= 0) & (pg < kn.shape[0])]
        if len(t) == 0:
            assert (got_o[r] == 0).all() and np.isneginf(got_l[r]).all(), f"{what} request {r} sees nothing"
            continue
        kk, vv = kn[pg, t % page], vn[pg, t % page]
        for h in range(Hq):
            ds = (d + 4) * 2.0 ** -23 * sc * (np.abs(kk[:, h // G]) @ np.abs(qn[r, h])).max()
            steps = (len(t) / 16 + 64) * 2.0 ** -23
            tol = np.abs(vv[:, h // G]).max() * (2 * ds + 2.0 ** -21 + (2.0 ** -16 if dtype == "bf16" else 0) + steps)
            d_o = np.abs(got_o[r, h] - ref[r, h])
            lim = HALF[dtype] * np.abs(ref[r, h]) + tol
            assert (d_o <= lim).all(), f"{what} request {r} head {h}: {(d_o / lim).max()} x tol"
            # lse: the largest score's error, the sum's relative one, and two roundings of its own size
            assert abs(got_l[r, h] - ref_lse[r, h]) <= ds + 2.0 ** -21 + steps + 2.0 ** -22 * abs(ref_lse[r, h]), f"{what} lse {r} {h}"


@pytest.mark.parametrize("dtype", ("f32", "bf16"))
@pytest.mark.parametrize("d", (64, 128))
@pytest.mark.parametrize("Hq,Hk,page", ((1, 1, 16), (8, 2, 16), (5, 1, 7), (16, 1, 64), (12, 4, 1), (40, 2, 32), (6, 6, 128)))
def test_attn_decode(dtype, d, Hq, Hk, page):
    lens = [1, 0, 15, 16, 17, 63, 64, 65, 200, 0, 333, 2]
    kc, vc, table = _cache(dtype, lens, page, Hk, d, seed=Hq + page + d)
    q = _randn(_rng(4), len(lens), Hq, d, dtype=dtype, scale=2.0)
    o, lse = binding.delta_rule_attn_decode(q, kc, vc, table, _i32(lens), want_lse=True)
    torch.cuda.synchronize()
    _check_attn(o, lse, q, kc, vc, table, lens, dtype)
    o2, none = binding.delta_rule_attn_decode(q, kc, vc, table, _i32(lens))
    torch.cuda.synchronize()
    assert none is None and torch.equal(o, o2)


@pytest.mark.parametrize("dtype", ("f32", "bf16"))
@pytest.mark.parametrize("lens,Hq,Hk", (([9000], 4, 1), ([1], 8, 8), ([0], 2, 1), ([0, 0, 0], 2, 2), ([5000, 3, 4097], 6, 2),
                                        ([700] * 40, 8, 4)))
def test_attn_decode_splits(dtype, lens, Hq, Hk):
    """Requests cut over many CTAs, requests that share one, and none at all; joint key-value pages."""
    kc, vc, table = _cache(dtype, lens, 16, Hk, 128, seed=len(lens), joint=True)
    q = _randn(_rng(5), len(lens), Hq, 128, dtype=dtype, scale=2.0)
    o, lse = binding.delta_rule_attn_decode(q, kc, vc, table, _i32(lens), want_lse=True)
    torch.cuda.synchronize()
    _check_attn(o, lse, q, kc, vc, table, lens, dtype)
    for _ in range(3):  # the split is joined in order: bit for bit
        o2, l2 = binding.delta_rule_attn_decode(q, kc, vc, table, _i32(lens), want_lse=True)
        assert torch.equal(o, o2) and torch.equal(lse, l2)


@pytest.mark.parametrize("dtype", ("f32", "bf16"))
def test_attn_decode_many_requests(dtype):
    """More requests than threads of a block, most of them of a tile or less: several share every block."""
    lens = [(7 * i) % 23 for i in range(777)]
    lens[400] = 1500
    kc, vc, table = _cache(dtype, lens, 8, 1, 64, seed=41)
    q = _randn(_rng(9), 777, 2, 64, dtype=dtype, scale=2.0)
    o, lse = binding.delta_rule_attn_decode(q, kc, vc, table, _i32(lens), want_lse=True)
    torch.cuda.synchronize()
    _check_attn(o, lse, q, kc, vc, table, lens, dtype)


@pytest.mark.parametrize("dtype", ("f32", "bf16"))
@pytest.mark.parametrize("page", (5, 32))
def test_attn_decode_caches_of_different_strides(dtype, page):
    lens = [100, 3, 64]
    kc, vc, table = _cache(dtype, lens, page, 2, 128, seed=page)
    P = kc.shape[0]
    kb = torch.full((P, 2, *kc.shape[1:]), float("nan"), dtype=DT[dtype], device="cuda")
    vb = torch.full((P, 3, *kc.shape[1:]), float("nan"), dtype=DT[dtype], device="cuda")
    kb[:, 1], vb[:, 2] = kc, vc
    q = _randn(_rng(9), 3, 10, 128, dtype=dtype)
    want = binding.delta_rule_attn_decode(q, kc, vc, table, _i32(lens), want_lse=True)
    got = binding.delta_rule_attn_decode(q, kb[:, 1], vb[:, 2], table, _i32(lens), want_lse=True)
    torch.cuda.synchronize()
    _check_attn(*want, q, kc, vc, table, lens, dtype)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    # heads before tokens; heads before pages, in one of the two; a slice of more heads
    hnd = lambda t: t.permute(0, 2, 1, 3).contiguous().permute(0, 2, 1, 3)  # noqa: E731
    first = vc.permute(2, 0, 1, 3).contiguous().permute(1, 2, 0, 3)
    wide = torch.full((P, page, 5, 128), float("nan"), dtype=DT[dtype], device="cuda")
    wide[:, :, 2:4] = kc
    for k2, v2 in ((hnd(kc), hnd(vc)), (kc, first), (wide[:, :, 2:4], hnd(vc))):
        got = binding.delta_rule_attn_decode(q, k2, v2, table, _i32(lens), want_lse=True)
        torch.cuda.synchronize()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_attn_decode_without_pages_or_table():
    q = _randn(_rng(9), 3, 4, 64, dtype="bf16")
    none = torch.empty(0, 16, 2, 64, dtype=torch.bfloat16, device="cuda")
    kc = torch.zeros(2, 16, 2, 64, dtype=torch.bfloat16, device="cuda")
    for cache, table in ((none, _i32([[0, 1]] * 3)), (kc, torch.empty(3, 0, dtype=torch.int32, device="cuda"))):
        o, lse = binding.delta_rule_attn_decode(q, cache, cache, table, _i32([5, 0, 40]), want_lse=True)
        torch.cuda.synchronize()
        assert (o == 0).all() and torch.isneginf(lse).all()
    o, lse = binding.delta_rule_attn_decode(q[:0], kc, kc, _i32([[0]])[:0], _i32([0])[:0], want_lse=True)
    assert o.shape == (0, 4, 64) and lse.shape == (0, 4)


@pytest.mark.parametrize("dtype", ("f32", "bf16"))
@pytest.mark.parametrize("window", (1, 2, 16, 33, 100, 5000))
def test_attn_decode_window(dtype, window):
    lens = [1, 0, 16, 31, 99, 100, 101, 400]
    kc, vc, table = _cache(dtype, lens, 7, 2, 64, seed=window)
    for r, n in enumerate(lens):  # what the window hides may be anything
        for t in range(max(0, n - window)):
            kc[table[r, t // 7], t % 7] = float("inf")
            vc[table[r, t // 7], t % 7] = float("nan")
    q = _randn(_rng(6), len(lens), 6, 64, dtype=dtype)
    o, lse = binding.delta_rule_attn_decode(q, kc, vc, table, _i32(lens), window=window, want_lse=True)
    torch.cuda.synchronize()
    _check_attn(o, lse, q, kc, vc, table, lens, dtype, window=window)


@pytest.mark.parametrize("dtype", ("f32", "bf16"))
def test_attn_decode_bad_pages_and_lengths(dtype):
    """Entries that are no page, lengths below zero and behind the table: not seen, and nothing of them read."""
    lens = [100, 48, 64, 33, 20]
    kc, vc, table = _cache(dtype, lens, 16, 2, 128, seed=3)
    table[0, 2], table[0, 3], table[1, :] = -1, 10 ** 6, -5
    table[2, 0] = kc.shape[0]
    told = [100, 48, 10 ** 6, -4, 2 ** 31 - 1]
    for r in (2, 4):  # the whole table's width is seen: fill its rows
        for j in range(table.shape[1]):
            if table[r, j] < 0:
                table[r, j] = table[3, 0]
    kc[kc.isnan()] = 0.5
    vc[vc.isnan()] = 0.25
    q = _randn(_rng(7), 5, 4, 128, dtype=dtype)
    o, lse = binding.delta_rule_attn_decode(q, kc, vc, table, _i32(told), want_lse=True)
    torch.cuda.synchronize()
    _check_attn(o, lse, q, kc, vc, table, told, dtype)


@pytest.mark.parametrize("dtype", ("f32", "bf16"))
def test_attn_decode_scales_and_extreme_scores(dtype):
    """A maximum that keeps rising, one far above the rest, scale 0 and below 0, and infinities."""
    lens = [200, 130]
    kc, vc, table = _cache(dtype, lens, 16, 1, 64, seed=11)
    q = torch.ones(2, 3, 64, dtype=DT[dtype], device="cuda")
    for t in range(200):  # scores rise by 1/4 a token
        kc[table[0, t // 16], t % 16] = t / 256.0
    kc[table[1, 3], 5] = 40.0  # a score of 320
    for scale in (None, 0.0, -0.125, 1.0):
        o, lse = binding.delta_rule_attn_decode(q, kc, vc, table, _i32(lens), scale=scale, want_lse=True)
        torch.cuda.synchronize()
        _check_attn(o, lse, q, kc, vc, table, lens, dtype, scale=scale, what=f"scale {scale}")
    kc[table[0, 0], 3] = float("-inf")  # never chosen; its value does not matter
    o, lse = binding.delta_rule_attn_decode(q, kc, vc, table, _i32(lens), want_lse=True)
    torch.cuda.synchronize()
    _check_attn(o, lse, q, kc, vc, table, lens, dtype, what="a score of -inf")
    kc[table[0, :5].long()] = float("-inf")  # every visible score is -inf: as a request that sees nothing
    o, lse = binding.delta_rule_attn_decode(q, kc, vc, table, _i32([70, 130]), want_lse=True)
    torch.cuda.synchronize()
    assert (o[0] == 0).all() and torch.isneginf(lse[0]).all() and o[1].isfinite().all()
    vc[table[1, 2], 1] = float("nan")  # a visible NaN is not hidden, and stays in its request
    o, lse = binding.delta_rule_attn_decode(q, kc, vc, table, _i32(lens), want_lse=True)
    torch.cuda.synchronize()
    assert o[1].isnan().all() and not o[0].isnan().any()
    kc[table[1, 2], 1] = float("nan")
    o, lse = binding.delta_rule_attn_decode(q, kc, vc, table, _i32(lens), want_lse=True)
    torch.cuda.synchronize()
    assert o[1].isnan().all() and lse[1].isnan().all() and not o[0].isnan().any()


def test_attn_decode_offsets_behind_2_to_31():
    """Rows whose element offset passes 2^31 and whose byte offset passes 2^32."""
    page, Hk, d = 64, 8, 128
    P = 2 ** 31 // (page * Hk * d) + 40
    kc = torch.empty(P, page, Hk, d, dtype=torch.bfloat16, device="cuda")
    vc = torch.empty(P, page, Hk, d, dtype=torch.bfloat16, device="cuda")
    table = _i32([[P - 1, 0, P - 2], [P - 3, 1, P // 2]])
    g = _rng(1)
    for p in table.flatten().tolist():
        kc[p], vc[p] = _randn(g, page, Hk, d, dtype="bf16"), _randn(g, page, Hk, d, dtype="bf16")
    q = _randn(g, 2, 16, d, dtype="bf16")
    lens = _i32([150, 192])
    o, lse = binding.delta_rule_attn_decode(q, kc, vc, table, lens, want_lse=True)
    rows = torch.cat([table[0], table[1]]).long()
    small = _i32([[0, 1, 2], [3, 4, 5]])
    o2, lse2 = binding.delta_rule_attn_decode(q, kc[rows].contiguous(), vc[rows].contiguous(), small, lens, want_lse=True)
    torch.cuda.synchronize()
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    _check_attn(o, lse, q, kc[rows], vc[rows], small, [150, 192], "bf16")
    # and into such rows
    slots = torch.tensor([(P - 1) * page + 5, 3], device="cuda")
    x = _randn(g, 2, 16 + 2 * Hk, d, dtype="bf16")
    f, pos = _freq(128), _i32([9, 8])
    binding.delta_rule_qkrope_cache(x[:, :16], x[:, 16:16 + Hk], x[:, 16 + Hk:], None, None, f, pos, slots, kc, vc)
    want = binding.delta_rule_qkrope(x[:, :16], x[:, 16:16 + Hk], None, None, f, pos)[1]
    torch.cuda.synchronize()
    assert torch.equal(kc[P - 1, 5], want[0]) and torch.equal(kc[0, 3], want[1]) and torch.equal(vc[P - 1, 5], x[0, 16 + Hk:])


def test_attn_decode_streams_and_graphs():
    """Two streams at once, each with its own workspace, and a captured call replayed with new lengths."""
    lens = [3000, 40, 0, 700]
    kc, vc, table = _cache("bf16", lens, 16, 2, 128, seed=21)
    q = _randn(_rng(8), 4, 8, 128, dtype="bf16")
    ln = _i32(lens)
    want, want_l = binding.delta_rule_attn_decode(q, kc, vc, table, ln, want_lse=True)
    torch.cuda.synchronize()
    got = []
    streams = [torch.cuda.Stream() for _ in range(2)]
    for i in range(6):
        with torch.cuda.stream(streams[i % 2]):
            got.append(binding.delta_rule_attn_decode(q, kc, vc, table, ln, want_lse=True))
    torch.cuda.synchronize()
    assert all(torch.equal(a, want) and torch.equal(b, want_l) for a, b in got)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, lse = binding.delta_rule_attn_decode(q, kc, vc, table, ln, want_lse=True)
    for new in ([3000, 40, 0, 700], [17, 0, 0, 699], [0, 0, 0, 0], [2999, 1, 0, 2]):
        ln.copy_(_i32(new))
        graph.replay()
        torch.cuda.synchronize()
        _check_attn(o, lse, q, kc, vc, table, new, "bf16", what=f"replayed {new}")


def test_attn_decode_behind_copies_in_a_graph():
    """Copies and other libraries' kernels between the calls, eager and captured: every call sees what was
    enqueued before it, although its kernels are set up while those still run."""
    lens = [4000, 1, 900]
    kc, vc, table = _cache("bf16", lens, 16, 1, 128, seed=23)
    q1, q2 = _randn(_rng(1), 3, 4, 128, dtype="bf16"), _randn(_rng(2), 3, 4, 128, dtype="bf16")
    ln = _i32(lens)
    want = [binding.delta_rule_attn_decode(x, kc, vc, table, ln)[0].clone() for x in (q1, q2)]
    q, n = torch.zeros_like(q1), torch.zeros_like(ln)

    def step(src):
        n.zero_()
        q.fill_(7.0)
        q.copy_(src)                               # a copy node
        n.copy_(ln)
        o, _ = binding.delta_rule_attn_decode(q, kc, vc, table, n)
        return o * 1.0                             # another kernel behind it

    for _ in range(20):
        got = [step(q1), step(q2)]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = [step(q1), step(q2), step(q1)]
    for _ in range(5):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]) and torch.equal(got[2], want[0])


def test_captured_across_streams_and_replayed_at_once():
    """One capture that forks to a second stream and joins again, and two graphs replayed on two streams."""
    lens = [2500, 1, 60, 800]
    kc, vc, table = _cache("bf16", lens, 16, 2, 64, seed=25)
    q, ln = _randn(_rng(1), 4, 8, 64, dtype="bf16"), _i32(lens)
    x, k, _, (wq, wk), f, pos = _qk_case("bf16", 2, 300, 4, 2, 64, 64, seed=26)
    gq, gk = _randn(_rng(2), 2, 300, 4, 64, dtype="bf16"), _randn(_rng(3), 2, 300, 2, 64, dtype="bf16")

    def both(side):
        main = torch.cuda.current_stream()
        side.wait_stream(main)
        with torch.cuda.stream(side):
            o = binding.delta_rule_attn_decode(q, kc, vc, table, ln, want_lse=True)
        y = binding.delta_rule_qkrope(x, k, wq, wk, f, pos)
        g = binding.delta_rule_qkrope_bwd(x, k, wq, wk, f, gq, gk, pos)
        main.wait_stream(side)
        o2 = binding.delta_rule_attn_decode(q, kc, vc, table, ln, want_lse=True)  # behind both branches
        return (*o, *y, *g, *o2)

    want = [t.clone() for t in both(torch.cuda.Stream())]
    torch.cuda.synchronize()
    graphs, outs = [], []
    for _ in range(2):
        graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
        with torch.cuda.graph(graph):
            outs.append(both(side))
        graphs.append(graph)
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(4):
        for graph, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                graph.replay()
    torch.cuda.synchronize()
    for out in outs:
        assert all(torch.equal(a, b) for a, b in zip(out, want))


def test_attn_decode_given_buffers():
    lens = [70, 500]
    kc, vc, table = _cache("f32", lens, 16, 2, 64, seed=24)
    q = _randn(_rng(3), 2, 4, 64)
    want, _ = binding.delta_rule_attn_decode(q, kc, vc, table, _i32(lens))
    ws = torch.full((binding.load().delta_rule_attn_decode_workspace_size(4, 2, 64, binding.DR_F32),), 255,
                    dtype=torch.uint8, device="cuda")  # what it holds on entry does not matter
    out = torch.full_like(q, float("nan"))
    got, _ = binding.delta_rule_attn_decode(q, kc, vc, table, _i32(lens), out=out, workspace=ws)
    torch.cuda.synchronize()
    assert got.data_ptr() == out.data_ptr() and torch.equal(out, want)
    small = torch.empty(256, dtype=torch.uint8, device="cuda")  # too small: one is allocated
    assert torch.equal(binding.delta_rule_attn_decode(q, kc, vc, table, _i32(lens), workspace=small)[0], want)


def test_python_level_refusals_on_cuda_tensors():
    x = torch.zeros(4, 6, 64, device="cuda")
    k, f, pos = torch.zeros(4, 2, 64, device="cuda"), _freq(64), _i32([0, 1, 2, 3])
    w = torch.ones(64, device="cuda")
    kc = torch.zeros(5, 16, 2, 64, device="cuda")
    slots, table, lens = torch.zeros(4, dtype=torch.int64, device="cuda"), _i32([[0, 1]] * 4), _i32([3] * 4)
    ok = dict(q=x, k=k, wq=w, wk=w, inv_freq=f, positions=pos)
    binding.delta_rule_qkrope(**ok)
    for bad in (dict(q=x.half()), dict(k=k.bfloat16()), dict(k=k[:3]), dict(wq=w[:32]), dict(wk=w.double()), dict(inv_freq=f.float()),
                dict(positions=pos.long()), dict(positions=pos[:2]), dict(q=x.transpose(0, 1)), dict(k=k.cpu()), dict(wq=w.cpu()),
                dict(q=x[0]), dict(positions=_i32([0] * 8)[::2])):
        with pytest.raises(ValueError):
            binding.delta_rule_qkrope(**{**ok, **bad})
    for bad in (dict(inv_freq=f[:20]), dict(q=x[..., :32].contiguous(), k=k[..., :32].contiguous(), wq=None, wk=None, inv_freq=f[:16])):
        with pytest.raises(binding.DeltaRuleError) as e:
            binding.delta_rule_qkrope(**{**ok, **bad})
        assert e.value.code == binding.DR_ERR_UNSUPPORTED
    with pytest.raises(ValueError):
        binding.delta_rule_qkrope_bwd(x, k, w, w, f, x[:3], k, pos)
    with pytest.raises(ValueError):
        binding.delta_rule_qkrope_bwd(x, k, w, w, f, x, k, pos, dq=x.bfloat16())
    cache = dict(q=x, k=k, v=k, wq=w, wk=w, inv_freq=f, positions=pos, slots=slots, k_cache=kc, v_cache=kc.clone())
    binding.delta_rule_qkrope_cache(**cache)
    for bad in (dict(slots=slots.int()), dict(slots=slots[:2]), dict(positions=None), dict(v=x), dict(k_cache=kc[:, :8]),
                dict(v_cache=kc[:4]), dict(k_cache=kc.bfloat16()), dict(q_out=x.transpose(0, 1).contiguous().transpose(0, 1))):
        with pytest.raises(ValueError):
            binding.delta_rule_qkrope_cache(**{**cache, **bad})
    attn = dict(q=x, k_cache=kc, v_cache=kc, table=table, lens=lens)
    binding.delta_rule_attn_decode(**attn)
    for bad in (dict(q=x.bfloat16()), dict(table=table.long()), dict(table=table[:3]), dict(lens=lens[:3]), dict(lens=lens.long()),
                dict(q=x[:, :, ::2]), dict(k_cache=kc.transpose(1, 2)), dict(v_cache=kc[:3]), dict(out=x.bfloat16()),
                dict(workspace=x), dict(q=x[0]), dict(table=_i32([[0] * 4] * 4)[:, ::2]),
                dict(k_cache=torch.zeros(5, 16, 64, 2, device="cuda").transpose(2, 3))):
        with pytest.raises(ValueError):
            binding.delta_rule_attn_decode(**{**attn, **bad})
    for bad, want in ((dict(q=x[:, :5].contiguous()), binding.DR_ERR_ARG), (dict(window=-1), binding.DR_ERR_ARG)):
        with pytest.raises(binding.DeltaRuleError) as e:
            binding.delta_rule_attn_decode(**{**attn, **bad})
        assert e.value.code == want
    with pytest.raises(TypeError):
        binding.delta_rule_attn_decode(**{**attn, "scale": "a"})
    pages = dict(cached=lens, fresh=lens, free_pages=_i32([1, 2]), n_free=_i32([2]), table=table, page=16, tokens=12)
    for bad in (dict(cached=lens.long()), dict(fresh=lens[:2]), dict(n_free=_i32([1, 2])), dict(table=table[:2]), dict(tokens=-1),
                dict(table=table[0]), dict(free_pages=_i32([[1]]))):
        with pytest.raises(ValueError):
            binding.delta_rule_pages(**{**pages, **bad})
    with pytest.raises(binding.DeltaRuleError):
        binding.delta_rule_pages(**{**pages, "page": 0})
    for bad in (dict(tokens=2 ** 31 - 1), dict(cached=torch.zeros(8193, dtype=torch.int32, device="cuda"),
                                               fresh=torch.zeros(8193, dtype=torch.int32, device="cuda"),
                                               table=torch.zeros(8193, 1, dtype=torch.int32, device="cuda"))):
        before = torch.cuda.max_memory_reserved()
        with pytest.raises(binding.DeltaRuleError) as e:
            binding.delta_rule_pages(**{**pages, **bad})
        assert e.value.code == binding.DR_ERR_UNSUPPORTED and torch.cuda.max_memory_reserved() == before
    torch.cuda.synchronize()


# ------------------------------------------------------------------------------------ together
@pytest.mark.parametrize("dtype,page", (("bf16", 16), ("f32", 7)))
def test_serving_steps_together(dtype, page):
    """Prompts admitted, then decoding steps as one captured graph: pages, norm and rotation into the
    cache, attention -- against dense causal attention in fp64 over the same projections."""
    R, Hq, Hk, d, T = 5, 6, 2, 64, 60
    prompt = [17, 1, 40, 0, 16]
    steps = 9
    g = _rng(31)
    wq, wk, f = 1 + _randn(g, d, scale=0.3), 1 + _randn(g, d, scale=0.3), _freq(64)
    qkv = _randn(g, R, T, (Hq + 2 * Hk) * d, dtype=dtype, scale=1.5)

    def heads(x):
        return [y.unflatten(-1, (-1, d)) for y in x.split([Hq * d, Hk * d, Hk * d], -1)]

    F = R * (T // page + 2)
    kc = torch.zeros(F, page, Hk, d, dtype=DT[dtype], device="cuda")
    vc = torch.zeros_like(kc)
    table = torch.full((R, T // page + 2), -1, dtype=torch.int32, device="cuda")
    free = torch.randperm(F, generator=g).to(torch.int32).cuda()
    left, lens = _i32([F]), _i32([0] * R)
    # prompts, packed into one padded batch
    packed = torch.cat([qkv[r, :n] for r, n in enumerate(prompt)] + [qkv[0, :3]])
    new, cu, pos, slots, n_left = binding.delta_rule_pages(lens, _i32(prompt), free, left, table, page, packed.shape[0])
    q, k, v = heads(packed)
    binding.delta_rule_qkrope_cache(q, k, v, wq, wk, f, pos, slots, kc, vc)
    lens.copy_(new)
    left.copy_(n_left)
    # one step: request 3 stays empty
    fresh = _i32([1, 1, 1, 0, 1])
    x = torch.zeros(R, (Hq + 2 * Hk) * d, dtype=DT[dtype], device="cuda")  # the step's rows, packed
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        new, cu, pos, slots, n_left = binding.delta_rule_pages(lens, fresh, free, left, table, page, R)
        qs, ks, vs = heads(x)
        qo = binding.delta_rule_qkrope_cache(qs, ks, vs, wq, wk, f, pos, slots, kc, vc)
        # a request's query is its last row of the batch
        row = (cu[1:].long() - 1).clamp(min=0)
        o, lse = binding.delta_rule_attn_decode(qo[row], kc, vc, table, new, want_lse=True)
        lens.copy_(new)
        left.copy_(n_left)
    live = [0, 1, 2, 4]
    for i in range(steps):
        x.zero_()
        x[:4] = torch.stack([qkv[r, prompt[r] + i] for r in live])
        graph.replay()
        torch.cuda.synchronize()
        assert lens.tolist() == [n + (i + 1 if r != 3 else 0) for r, n in enumerate(prompt)]
        for r in live:
            n = prompt[r] + i + 1
            qd, kd, vd = (y[None] for y in heads(qkv[r, :n]))
            qr, kr = binding.delta_rule_qkrope(qd, kd, wq, wk, f)  # the training form: positions 0 .. n - 1
            one = _i32([[0]])
            kp, vp = kr.contiguous(), vd.contiguous()
            _check_attn(o[r:r + 1], lse[r:r + 1], qr[0, -1:], kp, vp, one, [n], dtype, what=f"step {i} request {r}")
        assert (o[3] == 0).all()

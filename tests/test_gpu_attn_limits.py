"""The softmax-attention layers' operators at the limits of their arithmetic, sizes and arguments:
what a comparison at ordinary inputs does not show.  Each tolerance is derived where it is used."""
import numpy as np
import pytest
import torch

from gated_delta_rule_107_b200 import binding
from oracle import attn as oa
from parity_util import np64
from test_gpu_attn import DT, HALF, _check_attn, _i32

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------------------------ attention
@pytest.mark.parametrize("dtype", ("f32", "bf16"))
@pytest.mark.parametrize("d,Hq,Hk,tiles", ((64, 3, 1, 1), (128, 3, 1, 1), (128, 12, 1, 40), (64, 32, 2, 40)))
def test_attn_decode_weights_keep_32_bits(dtype, d, Hq, Hk, tiles):
    """Values that cancel, so that the output is what the weights' rounding leaves.

    Of every 16 tokens 14 have the score -5/4 and the value 1, two the score 0 and values whose sum is
    minus what the 14 weights add up to.  e^-1.25 as a sum of two bf16 numbers would be off by 2^-17.2.
    In 32 bits: the score in base 2 is off by 2.25 x 2^-24 (scale log2 e and the product, rounded), so
    the weight by 2^-23.3, and by the exponential's 2^-22: together 2^-21.5; 16 addends, each cut or
    rounded at 2^-24 of the largest, 2^-20; all relative to the sum of the 14.  The tiles' sums cancel
    each for itself, so their errors add up as their weights do, and the ratio stays."""
    n = 16 * tiles
    p = np.exp(-1.25)
    x1 = torch.tensor(14 * p, dtype=torch.bfloat16)
    x2 = torch.tensor(14 * p - x1.double().item(), dtype=torch.bfloat16)
    kc, vc = (torch.zeros(tiles, 16, Hk, d, dtype=DT[dtype], device="cuda") for _ in range(2))
    q = torch.zeros(1, Hq, d, dtype=DT[dtype], device="cuda")
    q[..., 0] = 1.0
    kc[:, :, :, 0] = -1.25
    vc[:] = 1.0
    kc[:, 5], kc[:, 11] = 0.0, 0.0
    vc[:, 5], vc[:, 11] = -x1.item(), -x2.item()
    table = torch.arange(tiles, dtype=torch.int32, device="cuda")[None]
    o, lse = binding.delta_rule_attn_decode(q, kc, vc, table, _i32([n]), scale=1.0, want_lse=True)
    torch.cuda.synchronize()
    ref, ref_lse = oa.attn_decode(np64(q), np64(kc), np64(vc), table.cpu().numpy(), [n], 1.0)
    tol = 14 * p / (14 * p + 2) * (2.0 ** -21.5 + 2.0 ** -20) + HALF[dtype] * np.abs(ref)
    worst = (np.abs(np64(o) - ref) / tol).max()
    assert worst <= 1, f"{worst} x tol"
    assert np.abs(np64(lse) - ref_lse).max() <= 2.0 ** -20 + (n / 16 + 8) * 2.0 ** -23


@pytest.mark.parametrize("d,Hq", ((128, 3), (64, 12)))
def test_attn_decode_long_sums_are_rounded_not_cut(d, Hq):
    """A long sum of one sign, and at its end values that cancel it: what is left is the sum's error.

    A warp adds up to 128 tiles.  Sums that are cut, not rounded, lose half a unit of the sum every
    time: with 384 additions of a third of a tile's product 2^-17 of the whole.  Rounded to nearest, the
    128 errors have no sign of their own: their standard deviation is 0.94 2^-23 of the whole for four
    warps (a uniform error of the growing sum's last place each, the sum of 4 warps' variances), of which
    six are allowed, 2^-20.5.  Besides: the weights' 2^-21.6 (score in base 2 off by 2^-23, the
    exponential by 2^-22), what is cut inside a tile's three products, 3 x 2^-23 of the tile's sum, and
    2^-22 for the last addition and the join."""
    R, tiles = 300, 512
    n, g = 16 * tiles, torch.Generator().manual_seed(d)
    score = -torch.randint(0, 65, (n,), generator=g).double() / 64
    score[::16] = 0.0
    value = (1 + torch.randint(0, 128, (n, d), generator=g).double() / 128)
    last = [n - 16, n - 13, n - 10]
    score[last] = 0.0
    value[last] = 0.0
    p = score.exp()
    left = (p[:, None] * value).sum(0)
    whole = left.clone()
    for t in last:
        value[t] = -left.bfloat16().double()
        left += value[t]
    kc, vc = (torch.zeros(tiles, 16, 1, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    kc.view(n, d)[:, 0] = score.bfloat16().cuda()
    vc.view(n, d).copy_(value.bfloat16())
    q = torch.zeros(R, Hq, d, dtype=torch.bfloat16, device="cuda")
    q[..., 0] = 1.0
    table = torch.arange(tiles, dtype=torch.int32, device="cuda").expand(R, tiles).contiguous()
    o, _ = binding.delta_rule_attn_decode(q, kc, vc, table, _i32([n] * R), scale=1.0)
    torch.cuda.synchronize()
    want = (left / p.sum()).numpy()
    tol = (whole / p.sum()).numpy() * (2.0 ** -20.5 + 2.0 ** -21.6 + 3 * 2.0 ** -23 + 2.0 ** -22) + HALF["bf16"] * np.abs(want)
    worst = (np.abs(np64(o) - want) / tol).max()
    assert worst <= 1, f"{worst} x tol"


@pytest.mark.parametrize("dtype", ("f32", "bf16"))
@pytest.mark.parametrize("d,Hq,Hk", ((64, 2, 1), (128, 3, 1), (128, 12, 1), (64, 32, 2), (128, 8, 8)))
def test_attn_decode_visible_infinities(dtype, d, Hq, Hk):
    """A value that is infinite and seen makes its channel infinite, whatever its weight; both signs
    together make NaN; other channels, heads and requests keep their numbers."""
    inf = float("inf")
    lens = [1, 3000, 3000, 700, 40]
    page, width = 16, 188
    g = torch.Generator().manual_seed(d + Hq)
    P = len(lens) * width
    kc, vc = (torch.randn(P, page, Hk, d, generator=g).to(DT[dtype]).cuda() for _ in range(2))
    q = torch.randn(len(lens), Hq, d, generator=g).to(DT[dtype]).cuda()
    table = torch.arange(P, dtype=torch.int32, device="cuda").view(len(lens), width)
    lens_t = _i32(lens)
    plain, lse = binding.delta_rule_attn_decode(q, kc, vc, table, lens_t, want_lse=True)
    want = plain.clone()

    def put(r, t, h, ch, x):
        vc[table[r, t // page], t % page, h, ch] = x
        heads = slice(h * (Hq // Hk), (h + 1) * (Hq // Hk))
        want[r, heads, ch] = torch.where(want[r, heads, ch] == -x, torch.full_like(want[r, heads, ch], float("nan")),
                                         torch.full_like(want[r, heads, ch], x))

    put(0, 0, 0, 3, inf)                       # one token: its weight is 1
    put(0, 0, Hk - 1, d - 1, -inf)
    for t in (0, 1, 17, 1500, 2999):           # weights with a rest of either sign; early ones are scaled down later
        put(1, t, 0, (5 * t) % d, inf)
    put(2, 100, 0, 7, inf)                     # both signs: NaN
    put(2, 2500, 0, 7, -inf)
    put(3, 699, Hk - 1, 0, -inf)
    vc[table[4, 2], 8, 0, 5] = inf             # token 40: not seen
    o, lse2 = binding.delta_rule_attn_decode(q, kc, vc, table, lens_t, want_lse=True)
    torch.cuda.synchronize()
    assert torch.equal(lse, lse2)
    assert torch.equal(o.isnan(), want.isnan()) and torch.equal(o.nan_to_num(nan=0.0), want.nan_to_num(nan=0.0))


@pytest.mark.parametrize("dtype", ("f32", "bf16"))
def test_attn_decode_infinity_of_no_noticeable_weight(dtype):
    """An infinite value whose score lies 300 below the largest, seen before it, after it and beside it."""
    d, n = 64, 2000
    kc, vc = (torch.zeros(n // 16, 16, 1, d, dtype=DT[dtype], device="cuda") for _ in range(2))
    q = torch.zeros(1, 2, d, dtype=DT[dtype], device="cuda")
    q[..., 0] = 1.0
    vc[:] = 0.5
    k = kc.view(n, d)
    table = torch.arange(n // 16, dtype=torch.int32, device="cuda")[None]
    for top in (0, 3, 1000, n - 1):
        k[:, 0] = -300.0
        k[top, 0] = 0.0
        for t in (1, 2, 14, 999, 1001, n - 2):
            vc.view(n, d)[t, 9] = float("inf")
            o, lse = binding.delta_rule_attn_decode(q, kc, vc, table, _i32([n]), scale=1.0, want_lse=True)
            torch.cuda.synchronize()
            vc.view(n, d)[t, 9] = 0.5
            assert (o[..., 9] == float("inf")).all(), (top, t)
            assert (o[..., :9] == 0.5).all() and (lse.abs() <= 2.0 ** -21).all(), (top, t)


# ------------------------------------------------------------------------------------ pages
SIZES = """
import sys
import torch
from gated_delta_rule_107_b200 import binding
from oracle import attn as oa
each = int(sys.argv[1])
for R in (4074, 4075, 4090, 4095, 4096):
    cached = torch.arange(R, dtype=torch.int32) % 5
    fresh = torch.full((R,), each, dtype=torch.int32)
    fresh[::3] = 0
    page, N = 4, int(fresh.sum()) + 3
    width = (4 + each) // page + 1
    table = torch.full((R, width), -1, dtype=torch.int32)
    table[:, :2] = torch.arange(2 * R, dtype=torch.int32).view(R, 2)
    free = torch.arange(R * width, dtype=torch.int32) + 2 * R
    want = oa.pages(cached.numpy(), fresh.numpy(), free.numpy(), len(free), table.numpy(), page, N)
    t = table.cuda()
    got = binding.delta_rule_pages(cached.cuda(), fresh.cuda(), free.cuda(),
                                   torch.tensor([len(free)], dtype=torch.int32, device="cuda"), t, page, N) + (t,)
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert (a.cpu().long() == torch.as_tensor(b).long()).all(), R
"""


@pytest.mark.parametrize("each", (1, 16))
def test_pages_of_thousands_of_requests_in_a_fresh_process(each):
    """Prefix sums around the shared memory that a kernel has unasked, with no larger call before them;
    few tokens, and so many that a lane takes several."""
    import subprocess
    import sys

    from conftest import ROOT
    r = subprocess.run([sys.executable, "-c", SIZES, str(each)], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]


@pytest.mark.parametrize("dtype", ("f32", "bf16"))
@pytest.mark.parametrize("told,window,seen", ((74, 16, range(58, 64)), (80, 16, ()), (79, 16, (63,)), (2 ** 31 - 1, 2 ** 31 - 60, range(59, 64)),
                                              (2 ** 31 - 1, 5, ()), (64, 16, range(48, 64)), (100, 0, range(64))))
def test_attn_decode_window_counts_back_from_the_length(dtype, told, window, seen):
    """A length behind the table: of the window's tokens only those inside it are seen."""
    g = torch.Generator().manual_seed(1)
    kc, vc = (torch.randn(5, 16, 1, 64, generator=g).to(DT[dtype]).cuda() for _ in range(2))
    q = torch.randn(2, 2, 64, generator=g).to(DT[dtype]).cuda()
    table = _i32([[3, 0, 4, 1], [2, 1, 0, 3]])
    o, lse = binding.delta_rule_attn_decode(q, kc, vc, table, _i32([told, 20]), window=window, want_lse=True)
    torch.cuda.synchronize()
    seen = list(seen)
    if not seen:
        assert (o[0] == 0).all() and torch.isneginf(lse[0]).all()
        return
    k, v = (np64(c)[[3, 0, 4, 1]].reshape(64, 64)[seen] for c in (kc, vc))
    s = np64(q)[0] @ k.T / 8
    p = np.exp(s - s.max(-1, keepdims=True))
    want = p @ v / p.sum(-1, keepdims=True)
    # scores of 64 products in 32 bits, weights, sums: far below what a token more or less changes
    ds = 68 * 2.0 ** -23 * (np.abs(np64(q)[0]) @ np.abs(k).T).max() / 8
    tol = HALF[dtype] * np.abs(want) + np.abs(v).max() * (2 * ds + 2.0 ** -20 + 72 * 2.0 ** -23)
    assert (np.abs(np64(o)[0] - want) <= tol).all()
    assert np.abs(np64(lse)[0] - (s.max(-1) + np.log(p.sum(-1)))).max() <= ds + 2.0 ** -20 + 72 * 2.0 ** -23


# ------------------------------------------------------------------------------------ norm and rotation
@pytest.mark.parametrize("dtype", ("f32", "bf16"))
@pytest.mark.parametrize("interleaved", (False, True))
@pytest.mark.parametrize("d,rot", ((64, 0), (128, 64), (128, 96), (64, 16)))
def test_qkrope_infinity_in_a_channel_that_is_not_turned(dtype, interleaved, d, rot):
    """It stays in its channel: the row's others are divided by an infinite norm, and in the backward the
    weights' gradients of other channels are finite."""
    g = torch.Generator().manual_seed(d + rot)
    N = 8
    f = 100.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / d).cuda() if rot else None
    for c in (rot, rot + 5, d - 1, (rot + d) // 2):
        x, dy = (torch.randn(N, 2, d, generator=g).to(DT[dtype]).cuda() for _ in range(2))
        others = torch.arange(d, device="cuda") != c
        y = x.clone()
        y[3, 1, c] = float("inf")
        out, _ = binding.delta_rule_qkrope(y, x, None, None, f, interleaved=interleaved)
        plain, _ = binding.delta_rule_qkrope(x, x, None, None, f, interleaved=interleaved)
        dy2 = dy.clone()
        dy2[3, 1, c] = float("inf")
        dw = binding.delta_rule_qkrope_bwd(x, x, None, None, f, dy2, dy, interleaved=interleaved)[2:]
        torch.cuda.synchronize()
        assert (out[3, 1, others] == 0).all() and out[3, 1, c].isnan()
        plain[3, 1] = out[3, 1]
        assert torch.equal(out[:, :, others], plain[:, :, others])
        assert torch.equal(dw[0][others], dw[1][others]) and dw[0][c] == float("inf") * x[3, 1, c].item() and dw[1].isfinite().all()


@pytest.mark.parametrize("dtype", ("f32", "bf16"))
@pytest.mark.parametrize("N,d", ((1, 64), (5, 128), (9, 64)))
def test_qkrope_infinite_gradient_of_the_last_token(dtype, N, d):
    """Lanes behind the last token add nothing to the weights' gradients, whatever the last one's gradient is."""
    g = torch.Generator().manual_seed(N)
    x = torch.randn(N, 2, d, generator=g).to(DT[dtype]).cuda()
    dy = torch.randn(N, 2, d, generator=g).to(DT[dtype]).cuda()
    dy[-1, 1, 3] = float("inf")
    dw = binding.delta_rule_qkrope_bwd(x, x, None, None, None, dy, dy)[2:]
    torch.cuda.synchronize()
    want = dw[0].cpu().clone()
    want[3] = float("inf") * x[-1, 1, 3].item()  # the definition: the sum over rows of dy n
    for w in dw:
        assert w[torch.arange(d) != 3].isfinite().all() and torch.equal(w.cpu(), want)


@pytest.mark.parametrize("dtype,interleaved", (("f32", False), ("bf16", False), ("bf16", True)))
def test_qkrope_angles_keep_32_bits(dtype, interleaved):
    """The weights' gradients are fp32 whatever the inputs' type: for one row with the gradient 1 in the
    first channel of every pair they are n cos(angle) there and -n sin(angle) in the second.

    Rows of ones, so that n is one number, which position 0 gives as the kernel has it.  The angle's
    fraction of a turn is rounded once in [-1/2, 1/2], 2^-26 turns or 2^-23.3; a cosine to 32 bits is off
    by 2 units of 2^-24 more, the product by 2^-24 of itself: 2^-22 covers them."""
    d = 128
    x = torch.ones(1, 1, d, dtype=DT[dtype], device="cuda")
    ia, ib = (torch.arange(0, d, 2), torch.arange(1, d, 2)) if interleaved else (torch.arange(d // 2), torch.arange(d // 2, d))
    dy = torch.zeros_like(x)
    dy[0, 0, ia.cuda()] = 1.0
    f = 10000.0 ** (-torch.arange(0, d, 2, dtype=torch.float64) / d)
    pos = torch.tensor([0, 1, 2, 3, 5, 7, 50, 999] + [1000 + 37 * i for i in range(120)], dtype=torch.int32)
    got = torch.stack([binding.delta_rule_qkrope_bwd(x, x, None, None, f.cuda(), dy, dy, p.cuda().view(1), interleaved)[2]
                       for p in pos])
    torch.cuda.synchronize()
    got = got.cpu().double()
    n = got[0, ia[0]]
    angle = pos.double()[:, None] * f
    worst = max((got[:, ia] / n - angle.cos()).abs().max().item(), (got[:, ib] / n + angle.sin()).abs().max().item())
    assert abs(n - 1 / (1 + 1e-6) ** 0.5) <= 2.0 ** -22
    assert worst <= 2.0 ** -22, f"off by {worst * 2 ** 22} x 2^-22"


def test_pages_small_outputs_do_not_hold_the_large_ones():
    """n_left and lens are kept for the next step; the positions and slots of a large prefill are not."""
    R, N = 40, 300000
    cached, fresh = _i32([0] * R), _i32([N // R] * R)
    table = torch.full((R, N // R // 64 + 1), -1, dtype=torch.int32, device="cuda")
    free = torch.arange(table.numel(), dtype=torch.int32, device="cuda")
    lens, cu, pos, slots, left = binding.delta_rule_pages(cached, fresh, free, _i32([free.numel()]), table, 64, N)
    torch.cuda.synchronize()
    assert left.item() == free.numel() - R * -(-(N // R) // 64) and slots.numel() == pos.numel() == N
    for t in (lens, cu, left):
        assert t.untyped_storage().nbytes() <= 8 * R + 64
    few = binding.delta_rule_pages(cached, fresh, free, _i32([free.numel()]), table, 64, 100)  # all in one piece
    assert len({t.untyped_storage().data_ptr() for t in few}) == 1


def test_pages_of_neighbouring_buffers():
    """Buffers side by side in one allocation do not overlap; a table or a batch of no entries overlaps nothing."""
    R, F, width, page, N = 3, 9, 8, 4, 40
    mem = torch.zeros(4 * R + F + 3 + R * width + 4 + 3 * N + 8, dtype=torch.int32, device="cuda")
    at, where = 0, {}
    for name, n in (("slots", 2 * N), ("cached", R), ("fresh", R), ("free_pages", F), ("n_free", 1), ("table", R * width), ("lens", R),
                    ("cu_new", R + 1), ("positions", N), ("n_left", 1)):
        where[name] = mem[at:at + n]
        at += n
    cached, fresh = [7, 0, 30], [9, 12, 0]
    for name, v in (("cached", cached), ("fresh", fresh), ("free_pages", list(range(20, 20 + F))), ("n_free", [F])):
        where[name].copy_(_i32(v))
    order = ("cached", "fresh", "free_pages", "n_free", "table", "lens", "cu_new", "positions", "slots", "n_left")
    rc = binding.pages_raw(*(where[n].data_ptr() for n in order), R, F, width, page, N, torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    want = oa.pages(cached, fresh, list(range(20, 20 + F)), F, np.zeros((R, width)), page, N)
    assert rc == binding.DR_OK
    got = [where[n] for n in ("lens", "cu_new", "positions")] + [where["slots"].view(torch.int64), where["n_left"], where["table"].view(R, width)]
    for a, b in zip(got, want):
        assert (a.cpu().long() == torch.as_tensor(b).long()).all()
    where["table"] = where["cached"]  # no columns
    rc = binding.pages_raw(*(where[n].data_ptr() for n in order), R, F, 0, page, N, torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    assert rc == binding.DR_OK and (where["slots"].view(torch.int64) == -1).all()


@pytest.mark.parametrize("dtype", ("f32", "bf16"))
@pytest.mark.parametrize("d,Hq,Hk", ((64, 2, 1), (128, 12, 1), (64, 32, 2), (128, 8, 8)))
def test_attn_decode_values_without_weight(dtype, d, Hq, Hk):
    """Only scores of -inf: out = 0 and lse = -inf whatever the values hold, and such a part of a request
    adds nothing to the others."""
    lens = [40, 3000, 1]
    page, width = 16, 188
    g = torch.Generator().manual_seed(d)
    kc, vc = (torch.randn(3 * width, page, Hk, d, generator=g).to(DT[dtype]).cuda() for _ in range(2))
    q = torch.ones(3, Hq, d, dtype=DT[dtype], device="cuda")
    table = torch.arange(3 * width, dtype=torch.int32, device="cuda").view(3, width)
    for r in (0, 2):
        kc[table[r].long()] = float("-inf")
        vc[table[r].long()] = float("inf")
        vc[table[r].long(), 3, :, 5] = float("nan")
    k1, v1 = kc[table[1].long()].clone(), vc[table[1].long()].clone()
    kc[table[1, 10:120].long()] = float("-inf")  # finite values: nothing of them is seen
    o, lse = binding.delta_rule_attn_decode(q, kc, vc, table, _i32(lens), want_lse=True)
    short = torch.cat([table[1:2, :10], table[1:2, 120:]], 1).contiguous()
    kc[table[1].long()], vc[table[1].long()] = k1, v1
    torch.cuda.synchronize()
    for r in (0, 2):
        assert (o[r] == 0).all() and torch.isneginf(lse[r]).all(), r
    _check_attn(o[1:2], lse[1:2], q[1:2], kc, vc, short, [3000 - 110 * 16], dtype)


@pytest.mark.parametrize("dtype", ("f32", "bf16"))
def test_qkrope_cache_without_pages(dtype):
    """A cache of no pages, as the attention over it takes it: the queries come out, nothing is written."""
    g = torch.Generator().manual_seed(3)
    x = torch.randn(5, 6, 64, generator=g).to(DT[dtype]).cuda()
    none = torch.empty(0, 16, 2, 64, dtype=DT[dtype], device="cuda")
    pos, slots = _i32([0, 1, 2, 3, 4]), torch.tensor([-1, 0, 5, -1, 2 ** 40], device="cuda")
    f = 100.0 ** (-torch.arange(0, 64, 2, dtype=torch.float64) / 64).cuda()
    q = binding.delta_rule_qkrope_cache(x[:, :2], x[:, 2:4], x[:, 4:], None, None, f, pos, slots, none, none.clone())
    want, _ = binding.delta_rule_qkrope(x[:, :2], x[:, 2:4], None, None, f, pos)
    torch.cuda.synchronize()
    assert torch.equal(q, want)

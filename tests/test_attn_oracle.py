"""The fp64 reference of the softmax-attention operators (oracle/attn.py) against hand-worked
examples, identities and differences, and the entry points' refusals, without a GPU."""
import ctypes
import types

import numpy as np
import pytest

from oracle import attn as oa

RNG = np.random.default_rng


# ------------------------------------------------------------------------------------ the reference
def test_pages_hand_example():
    # pages of 4: request 0 has 3 tokens (page 7) and gets 3, request 1 starts with 5, request 2 rests
    table = [[7, -1, -1], [-1, -1, -1], [9, 9, 9]]
    lens, cu, pos, slots, left, t = oa.pages([3, 0, 4], [3, 5, 0], [11, 12, 13, 14], 4, table, 4, 10)
    assert lens.tolist() == [6, 5, 4] and cu.tolist() == [0, 3, 8, 8] and left == 1
    assert t.tolist() == [[7, 14, -1], [13, 12, -1], [9, 9, 9]]
    assert pos.tolist() == [3, 4, 5, 0, 1, 2, 3, 4, 0, 0]
    assert slots.tolist() == [31, 56, 57, 52, 53, 54, 55, 48, -1, -1]


def test_pages_short_stack_and_narrow_table():
    lens, _, pos, slots, left, t = oa.pages([0, 0], [5, 9], [3, 4], 2, [[-5, -5], [-5, -5]], 4, 14)
    assert left == -2 and t.tolist() == [[4, 3], [-1, -1]]  # request 1's pages are missing
    assert lens.tolist() == [5, 9] and slots[:5].tolist() == [16, 17, 18, 19, 12] and (slots[5:] == -1).all()
    assert pos[5:].tolist() == list(range(9))  # the ninth token is behind the table


@pytest.mark.parametrize("interleaved", (False, True))
@pytest.mark.parametrize("rot", (0, 4, 8))
def test_qkrope_identities(rot, interleaved):
    r = RNG(rot)
    x, f = r.standard_normal((5, 2, 8)), 10.0 ** -np.arange(rot // 2)
    pos = np.array([0, 1, 7, 100, 3])
    y = oa.qkrope(x, None, pos, f, interleaved)
    assert np.allclose((y * y).mean(-1), 1.0, atol=1e-5)                       # a rotation keeps the norm
    assert np.allclose(y[0], oa.qkrope(x, None, pos, f[:0])[0])                # position 0 turns nothing
    assert np.allclose(y[..., rot:], oa.qkrope(x, None, pos, f[:0])[..., rot:])
    z = oa.qkrope(np.repeat(x[:1], 5, 0), None, pos, f, interleaved)           # products depend on the distance
    z2 = oa.qkrope(np.repeat(x[:1], 5, 0), None, pos + 40, f, interleaved)
    assert np.allclose(np.einsum("nhd,mhd->nmh", z, z), np.einsum("nhd,mhd->nmh", z2, z2))


def test_qkrope_quarter_turn():
    x = np.array([[[3.0, 4.0, 0.0, 0.0]]])
    y = oa.qkrope(x, np.ones(4), [1], [np.pi / 2, 0.0], interleaved=True)  # (a, b) -> (-b, a)
    n = x / np.sqrt(25.0 / 4 + 1e-6)
    assert np.allclose(y, [[[-n[0, 0, 1], n[0, 0, 0], 0, 0]]])
    y = oa.qkrope(x, np.ones(4), [1], [0.0, np.pi / 2])                    # pairs (0, 2) and (1, 3)
    assert np.allclose(y, [[[n[0, 0, 0], 0, 0, n[0, 0, 1]]]])


@pytest.mark.parametrize("interleaved", (False, True))
def test_qkrope_gradient_against_differences(interleaved):
    r = RNG(3)
    x, w, dy = r.standard_normal((4, 2, 8)), 1 + 0.3 * r.standard_normal(8), r.standard_normal((4, 2, 8))
    f, pos = np.array([1.0, 0.1, 0.01]), np.array([0, 2, 5, 1000])
    dx, dw = oa.qkrope_bwd(x, w, pos, f, dy, interleaved)
    loss = lambda x_, w_: (dy * oa.qkrope(x_, w_, pos, f, interleaved)).sum()  # noqa: E731
    h = 1e-6
    for at in np.ndindex(x.shape):
        e = np.zeros_like(x)
        e[at] = h
        assert abs((loss(x + e, w) - loss(x - e, w)) / (2 * h) - dx[at]) < 1e-7
    for c in range(8):
        e = np.zeros(8)
        e[c] = h
        assert abs((loss(x, w + e) - loss(x, w - e)) / (2 * h) - dw[c]) < 1e-7


def test_attention_identities():
    r = RNG(5)
    page, Hk, d = 3, 2, 4
    kc, vc = r.standard_normal((6, page, Hk, d)), r.standard_normal((6, page, Hk, d))
    table = np.array([[4, 1, 5], [0, 2, -1], [3, 3, 3]])
    q = r.standard_normal((3, 4, d))
    o, lse = oa.attn_decode(q, kc, vc, table, [7, 1, 0])
    k = np.concatenate([kc[4], kc[1], kc[5]])[:7]
    v = np.concatenate([vc[4], vc[1], vc[5]])[:7]
    for h in range(4):  # heads 0, 1 share key head 0
        s = k[:, h // 2] @ q[0, h] / 2.0
        assert np.allclose(o[0, h], np.exp(s) @ v[:, h // 2] / np.exp(s).sum()) and np.isclose(lse[0, h], np.log(np.exp(s).sum()))
    assert np.allclose(o[1], vc[0, 0][[0, 0, 1, 1]])           # one token: its value
    assert (o[2] == 0).all() and np.isneginf(lse[2]).all()     # none: nothing
    ow, _ = oa.attn_decode(q, kc, vc, table, [7, 1, 0], window=1)
    assert np.allclose(ow[0], v[6][[0, 0, 1, 1]])
    ob, _ = oa.attn_decode(q, kc, vc, np.array([[9, 1, 5], [0, 2, -1], [3, 3, 3]]), [6, 5, 0])
    s = k[3:6, 0] @ q[0, 0] / 2.0                              # page 9 is no page: tokens 3 .. 5 remain
    assert np.allclose(ob[0, 0], np.exp(s) @ v[3:6, 0] / np.exp(s).sum())


# ------------------------------------------------------------------------------------ planted mistakes
PINS = ([test_pages_hand_example, test_pages_short_stack_and_narrow_table, test_qkrope_quarter_turn, test_attention_identities]
        + [lambda r=r, i=i: test_qkrope_identities(r, i) for r in (0, 4, 8) for i in (False, True)]
        + [lambda i=i: test_qkrope_gradient_against_differences(i) for i in (False, True)])
MUTANTS = [
    ("pages_from_the_bottom", "table[r, j] = free_pages[left] if left >= 0 else -1", "table[r, j] = free_pages[top - 1 - left] if left >= 0 else -1"),
    ("partial_page_dropped", "for j in range(min(ceil_div(a, page), width)", "for j in range(min(a // page, width)"),
    ("slot_without_row", "table[r, p // page] * page + p % page if ok", "table[r, p // page] * page if ok"),
    ("position_from_zero", "            positions.append(p)", "            positions.append(p - a)"),
    ("norm_without_root", "    y = x / np.sqrt((x * x).mean(-1, keepdims=True) + EPS)", "    y = x / ((x * x).mean(-1, keepdims=True) + EPS)"),
    ("sum_for_mean", "    y = x / np.sqrt((x * x).mean(-1, keepdims=True) + EPS)", "    y = x / np.sqrt((x * x).sum(-1, keepdims=True) + EPS)"),
    ("pairs_exchanged", "return (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)", "return (i, i + rot // 2) if interleaved else (2 * i, 2 * i + 1)"),
    ("turned_backwards", "a * c - b * s, b * c + a * s", "a * c + b * s, b * c - a * s"),
    ("gradient_not_turned_back", "np.asarray(dy, np.float64), positions, inv_freq, interleaved, -1.0)", "np.asarray(dy, np.float64), positions, inv_freq, interleaved, 1.0)"),
    ("gradient_without_projection", "(gn - n * (gn * n).mean(-1, keepdims=True)) / rms", "gn / rms"),
    ("weight_missing_in_gradient", "    gn = g if w is None else g * w\n", "    gn = g\n"),
    ("scale_missing", "s = scale * (k[:, h // G] @ q[r, h])", "s = k[:, h // G] @ q[r, h]"),
    ("group_of_heads", "s = scale * (k[:, h // G] @ q[r, h])", "s = scale * (k[:, h % Hk] @ q[r, h])"),
    ("window_ignored", "np.arange(max(0, n - window) if window else 0, n)", "np.arange(0, n)"),
    ("last_token_missing", "np.arange(max(0, n - window) if window else 0, n)", "np.arange(max(0, n - window) if window else 0, max(n - 1, 0))"),
    ("bad_page_seen", "ok = (pg >= 0) & (pg < n_pages)", "pg = pg % n_pages; ok = pg >= 0"),
    ("lse_without_maximum", "lse[r, h] = m + np.log(p.sum())", "lse[r, h] = np.log(p.sum())"),
]


@pytest.mark.parametrize("name,old,new", MUTANTS, ids=[m[0] for m in MUTANTS])
def test_mutant_is_caught(name, old, new, monkeypatch):
    src = open(oa.__file__).read()
    assert src.count(old) == 1, f"mutation site for {name}"
    mod = types.ModuleType(f"attn_{name}")
    exec(compile(src.replace(old, new), f"<{name}>", "exec"), mod.__dict__)
    monkeypatch.setitem(globals(), "oa", mod)
    caught = 0
    for pin in PINS:
        try:
            pin()
        except (AssertionError, ValueError, IndexError):
            caught += 1
    assert caught > 0, f"no pin catches {name}"


# ------------------------------------------------------------------------------------ refusals
@pytest.fixture(scope="module")
def lib():
    from gated_delta_rule_107_b200 import binding, build
    build.build()
    return binding.load()


A = 1 << 20  # an aligned address that is never read: every call below is refused before any launch


def test_pages_refusals(lib):
    from gated_delta_rule_107_b200 import binding as b
    ok = dict(cached=A, fresh=A, free_pages=A, n_free=A, table=A, lens=A, cu_new=A, positions=A, slots=A, n_left=A,
              R=4, F=8, width=2, page=16, N=4)

    def call(**kw):
        return b.pages_raw(*{**ok, **kw}.values(), None)

    for name in ("cached", "fresh", "free_pages", "n_free", "table", "lens", "cu_new", "positions", "slots", "n_left"):
        assert call(**{name: None}) == b.DR_ERR_ARG, name
        assert call(**{name: A + 2}) == b.DR_ERR_ALIGN, name
    assert call(slots=A + 4) == b.DR_ERR_ALIGN
    for bad in (dict(R=-1), dict(F=-1), dict(width=-1), dict(page=0), dict(N=-1)):
        assert call(**bad) == b.DR_ERR_ARG, bad
    assert call(R=8193) == b.DR_ERR_UNSUPPORTED and call(N=(1 << 30) + 1) == b.DR_ERR_UNSUPPORTED


def test_qkrope_refusals(lib):
    from gated_delta_rule_107_b200 import binding as b
    fwd = dict(q=A, k=A, wq=A, wk=A, inv_freq=A, positions=A, q_out=A, k_out=A, B=2, T=5, Hq=4, Hk=2, d=128, rot=128,
               interleaved=0, qs=1024, ks=1024, dtype=b.DR_BF16)
    bwd = dict(q=A, k=A, wq=A, wk=A, inv_freq=A, positions=A, dq_out=A, dk_out=A, dq=A, dk=A, dwq=A, dwk=A, B=2, T=5,
               Hq=4, Hk=2, d=128, rot=128, interleaved=0, qs=1024, ks=1024, dqs=1024, dks=1024, dtype=b.DR_BF16, ws=A,
               nws=1 << 30)
    cache = dict(q=A, k=A, v=A, wq=A, wk=A, inv_freq=A, positions=A, slots=A, q_out=A, kc=A, vc=A, N=5, Hq=4, Hk=2,
                 d=128, rot=128, interleaved=0, qs=1024, ks=1024, vs=1024, n_pages=3, page=16, kps=4096, kts=256, khs=128,
                 vps=4096, vts=256, vhs=128, dtype=b.DR_BF16)
    calls = ((fwd, b.qkrope_raw), (bwd, b.qkrope_bwd_raw), (cache, b.qkrope_cache_raw))
    for ok, fn in calls:
        def call(**kw):
            return fn(*{**ok, **kw}.values(), None)

        for name in set(ok) & {"q", "k", "v", "inv_freq", "slots", "q_out", "k_out", "dq_out", "dk_out", "dq", "dk", "kc", "vc"}:
            assert call(**{name: None}) == b.DR_ERR_ARG, name
            assert call(**{name: A + 4}) == b.DR_ERR_ALIGN, name
        for name in ("wq", "wk"):
            assert call(**{name: A + 4}) == b.DR_ERR_ALIGN, name
        assert call(positions=A + 1) == b.DR_ERR_ALIGN
        assert call(d=96) == b.DR_ERR_UNSUPPORTED and call(rot=24) == b.DR_ERR_UNSUPPORTED
        assert call(rot=256) == b.DR_ERR_ARG and call(rot=-16) == b.DR_ERR_ARG and call(interleaved=2) == b.DR_ERR_ARG
        assert call(dtype=7) == b.DR_ERR_ARG and call(Hq=-1) == b.DR_ERR_ARG
        assert call(Hq=1020, Hk=8) == b.DR_ERR_UNSUPPORTED
        for name in set(ok) & {"qs", "ks", "vs", "dqs", "dks", "kps", "kts", "khs", "vps", "vts", "vhs"}:
            assert call(**{name: 64}) == b.DR_ERR_ARG, name       # shorter than a token's heads, or a head
            assert call(**{name: 8196}) == b.DR_ERR_ALIGN, name   # rows off 16 bytes
    def wcall(**kw):
        return b.qkrope_bwd_raw(*{**bwd, **kw}.values(), None)
    need = lib.delta_rule_qkrope_workspace_size(128)
    assert need > 0 and lib.delta_rule_qkrope_workspace_size(96) == ctypes.c_size_t(-1).value
    assert wcall(ws=None) == b.DR_ERR_WORKSPACE and wcall(nws=need - 1) == b.DR_ERR_WORKSPACE
    assert wcall(ws=A + 16) == b.DR_ERR_ALIGN and wcall(dwq=A + 2) == b.DR_ERR_ALIGN
    assert b.qkrope_cache_raw(*{**cache, "page": 0}.values(), None) == b.DR_ERR_ARG
    assert b.qkrope_cache_raw(*{**cache, "Hk": 0}.values(), None) == b.DR_ERR_ARG
    assert b.qkrope_cache_raw(*{**cache, "positions": None}.values(), None) == b.DR_ERR_ARG
    assert b.qkrope_raw(*{**fwd, "T": 0}.values(), None) == b.DR_OK  # nothing to do
    assert b.qkrope_cache_raw(*{**cache, "N": 0}.values(), None) == b.DR_OK


def test_attn_decode_refusals(lib):
    from gated_delta_rule_107_b200 import binding as b
    ok = dict(q=A, kc=A, vc=A, table=A, lens=A, out=A, lse=A, R=2, Hq=8, Hk=2, d=128, n_pages=4, page=16, width=2,
              kps=4096, kts=256, khs=128, vps=4096, vts=256, vhs=128, scale=1.0, window=0, dtype=b.DR_BF16, ws=A, nws=1 << 30)

    def call(**kw):
        return b.attn_decode_raw(*{**ok, **kw}.values(), None)

    for name in ("q", "kc", "vc", "table", "lens", "out"):
        assert call(**{name: None}) == b.DR_ERR_ARG, name
    for name in ("q", "kc", "vc", "out"):
        assert call(**{name: A + 8}) == b.DR_ERR_ALIGN, name
    for name in ("table", "lens", "lse"):
        assert call(**{name: A + 2}) == b.DR_ERR_ALIGN, name
    for bad in (dict(R=-1), dict(Hq=0), dict(Hk=0), dict(Hq=7), dict(n_pages=-1), dict(page=0), dict(width=-1),
                dict(window=-1), dict(dtype=3), dict(kps=64), dict(vps=64), dict(kts=120), dict(vts=0), dict(khs=-128), dict(vhs=64)):
        assert call(**bad) == b.DR_ERR_ARG, bad
    assert call(d=96) == b.DR_ERR_UNSUPPORTED
    for name in ("kps", "kts", "khs", "vps", "vts", "vhs"):
        assert call(**{name: 4100}) == b.DR_ERR_ALIGN, name
    assert call(R=1 << 20, width=1 << 18, page=16) == b.DR_ERR_UNSUPPORTED
    need = lib.delta_rule_attn_decode_workspace_size(8, 2, 128, b.DR_BF16)
    assert call(ws=None) == b.DR_ERR_WORKSPACE and call(nws=need - 1) == b.DR_ERR_WORKSPACE
    assert call(ws=A + 16) == b.DR_ERR_ALIGN
    assert call(R=0) == b.DR_OK
    assert lib.delta_rule_attn_decode_workspace_size(7, 2, 128, b.DR_BF16) == ctypes.c_size_t(-1).value


def test_python_level_refusals():
    """Wrong element types, devices and layouts raise before the C call."""
    import torch

    from gated_delta_rule_107_b200 import binding as b
    x = torch.zeros(2, 3, 64)
    with pytest.raises(ValueError):
        b.delta_rule_qkrope(x, x)  # not CUDA tensors
    with pytest.raises(ValueError):
        b.delta_rule_attn_decode(x, x, x, x, x)
    with pytest.raises(ValueError):
        b.delta_rule_pages(x, x, x, x, x, 16, 4)
    tok, cs = b._calls().stride_of_tokens, b._calls().strides_of_cache
    assert tok(torch.zeros(5, 6 * 64).unflatten(-1, (6, 64))[:, 2:4]) == 384
    assert tok(torch.zeros(2, 5, 6, 64)[:, :, 1:3]) == 384
    assert tok(torch.zeros(2, 5, 6, 64)[:, :1]) == 5 * 384
    assert tok(torch.zeros(1, 1, 6, 64)) == tok(torch.zeros(3, 6, 64)[1:2]) == tok(torch.zeros(1, 7, 64)[:, :6]) == 384
    for bad in (torch.zeros(2, 5, 6, 64)[:, :3], torch.zeros(5, 64, 6).transpose(1, 2), torch.zeros(5, 6, 128)[..., ::2],
                torch.zeros(6, 64), torch.zeros(5, 6, 128)[..., :64]):
        with pytest.raises(ValueError):
            tok(bad)
    assert cs(torch.zeros(4, 2, 16, 2, 64)[:, 1]) == (2 * 16 * 2 * 64, 128, 64)
    assert cs(torch.zeros(1, 2, 16, 2, 64)[:, 1]) == (16 * 2 * 64, 128, 64)
    assert cs(torch.zeros(4, 2, 16, 64).transpose(1, 2)) == (2 * 16 * 64, 64, 16 * 64)  # heads first
    assert cs(torch.zeros(4, 16, 4, 64)[:, :, 1:3]) == (16 * 256, 256, 64)
    for bad in (torch.zeros(4, 16, 64), torch.zeros(4, 16, 2, 128)[..., ::2], torch.zeros(4, 16, 64, 2).transpose(2, 3)):
        with pytest.raises(ValueError):
            cs(bad)
    with pytest.raises(TypeError):
        tok(3)
    with pytest.raises(TypeError):
        b.delta_rule_qkrope(None, x)

"""The softmax-attention layers' reference, refusals and build at their limits, without a GPU."""
import numpy as np
import pytest

from oracle import attn as oa


def test_reference_window_counts_back_from_a_length_behind_the_table():
    """Eight rows of table, pages of 4: a length of 11 with a window of 5 sees tokens 6 and 7 of its 6 .. 10."""
    r = np.random.default_rng(2)
    kc, vc = r.standard_normal((2, 4, 1, 4)), r.standard_normal((2, 4, 1, 4))
    q, table = r.standard_normal((1, 1, 4)), np.array([[1, 0]])
    o, lse = oa.attn_decode(q, kc, vc, table, [11], window=5)
    s = kc[0, 2:4, 0] @ q[0, 0] / 2.0
    assert np.allclose(o[0, 0], np.exp(s) @ vc[0, 2:4, 0] / np.exp(s).sum()) and np.isclose(lse[0, 0], np.log(np.exp(s).sum()))
    for told, window in ((13, 5), (2 ** 31 - 1, 7)):  # the whole window lies behind
        o, lse = oa.attn_decode(q, kc, vc, table, [told], window=window)
        assert (o == 0).all() and np.isneginf(lse).all()
    o, _ = oa.attn_decode(q, kc, vc, table, [12], window=5)
    assert np.allclose(o[0, 0], vc[0, 3, 0])
    assert np.array_equal(oa.attn_decode(q, kc, vc, table, [99])[0], oa.attn_decode(q, kc, vc, table, [8])[0])


# ------------------------------------------------------------------------------------ refusals
@pytest.fixture(scope="module")
def binding():
    from gated_delta_rule_107_b200 import binding, build
    build.build()
    binding.load()
    return binding


def test_pages_refuses_outputs_that_overlap(binding):
    """Every block reads the lengths, the stack and its count while others write: an output that shares a
    byte with an input or another output is refused.  No address here is ever read."""
    R, F, width, page, N = 300, 500, 7, 16, 4000
    sizes = dict(cached=4 * R, fresh=4 * R, free_pages=4 * F, n_free=4, table=4 * R * width, lens=4 * R, cu_new=4 * (R + 1),
                 positions=4 * N, slots=8 * N, n_left=4)
    names = list(sizes)
    apart = {name: (i + 1) << 20 for i, name in enumerate(names)}

    def call(**kw):
        return binding.pages_raw(*{**apart, **kw}.values(), R, F, width, page, N, None)

    for out in ("table", "lens", "cu_new", "positions", "slots", "n_left"):
        for other in names:
            if other == out:
                continue
            at = apart[other]
            inside = at + (sizes[other] - 4) // 8 * 8          # the other's last whole word, or its only one
            before = at - (sizes[out] - 4) // 8 * 8            # the output's last words on the other's first
            for there in (at, inside, before):
                assert call(**{out: there}) == binding.DR_ERR_ARG, (out, other, there - at)


# ------------------------------------------------------------------------------------ the build
@pytest.fixture
def build(tmp_path, monkeypatch):
    """The build with compilers that only write what they were asked for, into a folder of its own."""
    from gated_delta_rule_107_b200 import build as b
    fake = tmp_path / "compiler"
    fake.write_text('#!/bin/sh\nall="$*"\necho "$all" >> ' + str(tmp_path / "calls") + '\nwhile [ "$1" != -o ]; do shift; done\n'
                    'echo "$all" > "$2"\n')
    fake.chmod(0o755)
    monkeypatch.setenv("NVCC", str(fake))
    monkeypatch.setenv("CXX", str(fake))
    monkeypatch.setattr(b, "LIB", str(tmp_path / "libdeltarule.so"))
    monkeypatch.setattr(b, "CALLS", str(tmp_path / "_torch_calls.so"))
    b.calls = lambda: (tmp_path / "calls").read_text().count("torch_calls.cpp") if (tmp_path / "calls").exists() else 0
    yield b
    del b.calls


def test_the_library_is_built_where_the_torch_module_cannot_be(build, monkeypatch, tmp_path):
    """libdeltarule.so needs nvcc and nothing else."""
    import os
    import subprocess
    import sys
    no = tmp_path / "no"
    no.write_text("#!/bin/sh\nexit 1\n")
    no.chmod(0o755)
    monkeypatch.setenv("CXX", str(no))
    with pytest.raises(subprocess.CalledProcessError):
        build.build(force=True)
    assert os.path.exists(build.LIB) and not os.path.exists(build.CALLS)
    os.remove(build.LIB)
    monkeypatch.setitem(sys.modules, "torch", None)  # importing it raises ImportError
    assert build.build(force=True) == build.LIB
    assert os.path.exists(build.LIB) and not os.path.exists(build.CALLS)


def test_the_torch_module_is_built_again_for_another_torch(build, monkeypatch):
    """File times do not show that torch, Python or the flags changed."""
    import torch
    build.build_calls()
    build.build_calls()
    assert build.calls() == 1
    monkeypatch.setattr(torch, "__version__", "9.9.9")
    build.build_calls()
    build.build_calls()
    assert build.calls() == 2

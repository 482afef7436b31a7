"""The paged cache and its attention without a GPU: refusals before any launch,
and the plain 64-bit implementations against brute force and invariants."""
import ctypes

import numpy as np
import pytest
import torch

import kv_ref as R
from speculative_decode_verify_gdn_amd import binding as gb

FAKE = ctypes.c_void_p(0x1000)  # never dereferenced: validation fails first
ODD = ctypes.c_void_p(0x1008)
OTHER = ctypes.c_void_p(0x2000)


@pytest.fixture(scope="module")
def lib():
    import os
    if not os.path.exists(gb.LIB_PATH):
        from speculative_decode_verify_gdn_amd import build
        build.build()
    return gb.lib()


def shape(**kw):
    d = dict(L=1, B=2, Hq=4, Hkv=2, D=64, page=16, n_pages=10, max_blocks=4)
    d.update(kw)
    return ctypes.byref(gb.KvShape(**d).c)


BAD_SHAPES = [
    (dict(L=0), 1), (dict(B=0), 1), (dict(Hq=0), 1), (dict(Hkv=0), 1), (dict(Hq=5), 1),
    (dict(n_pages=0), 1), (dict(max_blocks=0), 1), (dict(D=0), 1), (dict(page=0), 1),
    (dict(D=96), 2), (dict(D=32), 2), (dict(page=8), 2), (dict(page=24), 2), (dict(page=512), 2),
    (dict(n_pages=1 << 27), 2), (dict(max_blocks=(1 << 26) + 1), 2), (dict(B=65536), 2),
    (dict(L=32768), 2), (dict(Hq=65536, Hkv=1), 2), (dict(L=4096, B=4096), 2),
]


@pytest.mark.parametrize("kw,status", BAD_SHAPES)
def test_shapes_refused(lib, kw, status):
    sh = shape(**kw)
    assert lib.kv_reserve(sh, 1, 70000, FAKE, FAKE, FAKE, FAKE, FAKE, OTHER, FAKE, None, None) == status
    assert lib.kv_append(sh, 8, FAKE, 1024, FAKE, 1024, FAKE, FAKE, FAKE, None, None) == status
    assert lib.attn_verify(sh, 1, 70000, FAKE, FAKE, FAKE, None, FAKE, 1 << 20, 1.0, FAKE, FAKE, FAKE,
                           FAKE, 1 << 40, None, None) == status
    assert lib.kv_commit(sh, 1, 70000, FAKE, None, FAKE, None, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE,
                         FAKE, None, 0, None, 0, None, None, None, None) == status
    assert lib.attn_verify_workspace_bytes(sh, 1, 70000) == 0


def test_null_shape_refused(lib):
    assert lib.kv_append(None, 8, FAKE, 128, FAKE, 128, FAKE, FAKE, FAKE, None, None) == 1
    assert lib.attn_verify_workspace_bytes(None, 1, 1) == 0


def test_reserve_refusals(lib):
    good = [shape(), 4, 8, None, FAKE, FAKE, FAKE, FAKE, OTHER, FAKE, None, None]

    def call(**at):
        a = list(good)
        for k, v in at.items():
            a[int(k[1:])] = v
        return lib.kv_reserve(*a)

    for i in (4, 5, 6, 7, 8, 9):
        assert call(**{"a%d" % i: None}) == gb.GDN_ERR_INVALID_ARG
    assert call(a8=FAKE) == gb.GDN_ERR_INVALID_ARG          # n_left is n_free
    assert call(a1=0) == gb.GDN_ERR_INVALID_ARG
    assert call(a2=0) == gb.GDN_ERR_INVALID_ARG
    assert call(a2=7) == gb.GDN_ERR_INVALID_ARG             # 2 sequences of 4 need 8 rows
    assert call(a1=(1 << 24) + 1, a3=FAKE) == gb.GDN_ERR_UNSUPPORTED
    assert call(a2=(1 << 24) + 1) == gb.GDN_ERR_UNSUPPORTED


def test_append_refusals(lib):
    good = [shape(), 8, FAKE, 128, FAKE, 128, FAKE, FAKE, FAKE, None, None]

    def call(**at):
        a = list(good)
        for k, v in at.items():
            a[int(k[1:])] = v
        return lib.kv_append(*a)

    for i in (2, 4, 6, 7, 8):
        assert call(**{"a%d" % i: None}) == gb.GDN_ERR_INVALID_ARG
    for i in (2, 4, 7, 8):
        assert call(**{"a%d" % i: ODD}) == gb.GDN_ERR_INVALID_ARG
    for i in (3, 5):
        for ld in (127, 132, -128, 0, 1 << 40):
            assert call(**{"a%d" % i: ld}) == gb.GDN_ERR_INVALID_ARG
    assert call(a1=0) == gb.GDN_ERR_INVALID_ARG
    assert call(a1=(1 << 24) + 1) == gb.GDN_ERR_UNSUPPORTED


def test_attention_refusals(lib):
    ws = lib.attn_verify_workspace_bytes(shape(), 4, 8)
    assert ws > 0
    good = [shape(), 4, 8, None, FAKE, FAKE, None, FAKE, 256, 0.1, FAKE, FAKE, FAKE, FAKE, ws, None,
            None]

    def call(**at):
        a = list(good)
        for k, v in at.items():
            a[int(k[1:])] = v
        return lib.attn_verify(*a)

    for i in (4, 5, 7, 10, 11, 12):
        assert call(**{"a%d" % i: None}) == gb.GDN_ERR_INVALID_ARG
    for i in (7, 10, 11, 12):
        assert call(**{"a%d" % i: ODD}) == gb.GDN_ERR_INVALID_ARG
    for x in (float("nan"), float("inf"), -float("inf"), 3e38, -3e38):
        assert call(a9=x) == gb.GDN_ERR_INVALID_ARG
    assert call(a8=255) == gb.GDN_ERR_INVALID_ARG
    assert call(a8=260) == gb.GDN_ERR_INVALID_ARG
    assert call(a13=None) == gb.GDN_ERR_WORKSPACE
    assert call(a13=ODD) == gb.GDN_ERR_WORKSPACE
    assert call(a14=ws - 1) == gb.GDN_ERR_WORKSPACE
    assert call(a1=65, a2=130, a6=FAKE, a14=1 << 40) == gb.GDN_ERR_UNSUPPORTED  # a tree of 65
    assert call(a0=shape(Hq=256, Hkv=1), a2=1 << 23, a3=FAKE, a8=1 << 14,
                a14=1 << 40) == gb.GDN_ERR_UNSUPPORTED  # 2^31 rows of a key head
    assert lib.attn_verify_workspace_bytes(shape(), 0, 8) == 0
    assert lib.attn_verify_workspace_bytes(shape(), 4, 0) == 0


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_workspace_does_not_fall_with_the_tokens(lib, D, dtype):
    """A workspace made for the largest T, batch and n_tokens serves smaller calls."""
    for Hq in (1, 4, 7, 16, 70):
        sh = shape(Hq=Hq, Hkv=1, D=D, dtype=dtype)
        got = [lib.attn_verify_workspace_bytes(sh, T, 2 * T) for T in range(1, 300)]
        assert got[0] > 0 and all(a <= b for a, b in zip(got, got[1:]))
        assert got[-1] == lib.attn_verify_workspace_bytes(sh, 299, 10000)


def test_commit_refusals(lib):
    good = [shape(), 4, 8, None, None, FAKE, None, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, 128,
            FAKE, 128, FAKE, FAKE, None, None]

    def call(**at):
        a = list(good)
        for k, v in at.items():
            a[int(k[1:])] = v
        return lib.kv_commit(*a)

    for i in (5, 7, 8, 9, 10, 11, 12, 13):
        assert call(**{"a%d" % i: None}) == gb.GDN_ERR_INVALID_ARG
    for i in (14, 16, 18, 19):
        assert call(**{"a%d" % i: None, "a4": FAKE}) == gb.GDN_ERR_INVALID_ARG
        assert call(**{"a%d" % i: ODD, "a4": FAKE}) == gb.GDN_ERR_INVALID_ARG
    assert call(a4=FAKE, a15=64) == gb.GDN_ERR_INVALID_ARG
    assert call(a4=FAKE, a1=65, a2=130) == gb.GDN_ERR_UNSUPPORTED


def test_binding_refuses_host_and_odd_tensors():
    sh = gb.KvShape(1, 1, 2, 2, 64, 16, 4, 2)
    x = torch.zeros((1, 3, 2, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        gb._rows(x, "k", torch.bfloat16, (1, 3, 2, 64))      # host tensor
    with pytest.raises(TypeError):
        gb._rows(x, "k", torch.float32, (1, 3, 2, 64))
    with pytest.raises(ValueError):
        gb._rows(x, "k", torch.bfloat16, (1, 4, 2, 64))
    with pytest.raises(TypeError):
        gb.KvShape(1, 1, 2, 2, 64, 16, 4, 2, torch.float16).c
    assert sh.k_cache_shape == (1, 4, 2, 16, 64) and sh.v_cache_shape == (1, 4, 2, 2, 64, 8)


def _dense(bt, table, parent_of, scale):
    """The attention again, from dense masks over the whole batch at once."""
    sh, G = bt.sh, bt.sh.Hq // bt.sh.Hkv
    out = bt.o.astype(np.float64).copy()
    for b in range(sh.B):
        s, c = int(bt.q_start[b]), int(bt.seq_len[b])
        n = int(bt.q_start[b + 1]) - s
        rows = [table[b, j // sh.page] * sh.page + j % sh.page for j in range(c + n)]
        bias = np.full((n, c + n), -np.inf)
        bias[:, :c] = 0
        reach = np.eye(n)
        for v in range(n):
            p = parent_of(s, v)
            if p >= 0:
                reach[v] += reach[p]
        bias[:, c:][reach > 0] = 0
        for hq in range(sh.Hq):
            K = bt.kc.transpose(0, 1, 3, 2, 4).reshape(sh.L, -1, sh.Hkv, sh.D)[0, rows, hq // G]
            V = bt.vc.transpose(0, 1, 3, 5, 2, 4).reshape(sh.L, -1, sh.Hkv, sh.D)[0, rows, hq // G]
            z = scale * bt.q[0, s:s + n, hq].astype(np.float64) @ K.T.astype(np.float64) + bias
            e = np.exp(z)
            out[0, s:s + n, hq] = (e / e.sum(1, keepdims=True)) @ V.astype(np.float64)
    return out


@pytest.mark.parametrize("tree", [False, True])
def test_plain_attention_against_dense_masks(tree):
    bt = R.Batch(3, [0, 1, 17, 40], [1, 5, 0, 9], Hq=6, Hkv=2, tree=tree, pad=2, device=None,
                 dtype=torch.float32)
    table, slots, left, err = bt.r_reserve()
    kc, vc, e2 = bt.r_append(slots)
    assert err == 0 and e2 == 0
    bt.kc, bt.vc = kc, vc
    got, tol = bt.r_attend(table, kc, vc)
    want = _dense(bt, table, (lambda s, v: bt.parent[s + v]) if tree else (lambda s, v: v - 1),
                  bt.sh.D ** -0.5)
    np.testing.assert_allclose(got, want, rtol=0, atol=1e-12)
    assert (got[:, -2:] == 3.0).all() and (tol[:, -2:] == 0).all()


def _owned(sh, table, seq_len):
    return [int(p) for b in range(sh.B) for p in table[b, :R.up(int(seq_len[b]), sh.page)]]


def test_plain_pool_never_shares_a_page():
    """Rounds of reserve and commit with random lengths: every page is either on
    the stack or held by one sequence, and never both."""
    rng = np.random.default_rng(11)
    sh = gb.KvShape(1, 6, 2, 2, 64, 16, 16, 12)
    table = np.full((6, 12), -1, np.int64)
    free, n_free, ln = rng.permutation(16).astype(np.int64), 16, np.zeros(6, np.int64)
    kc, vc = np.zeros(sh.k_cache_shape, np.float32), np.zeros(sh.v_cache_shape, np.float32)
    seen = 0
    for _ in range(60):
        new = rng.integers(0, 30, 6)
        new = np.minimum(new, 12 * 16 - ln)
        start = np.concatenate([[0], np.cumsum(new)])
        N = max(1, int(start[-1]))
        table, slots, left, err = R.reserve(sh, 30, N, start, ln, table, free, n_free)
        seen |= err
        used = slots[slots >= 0]
        assert len(set(used.tolist())) == len(used)
        keep = np.array([rng.integers(0, n + 1) if n and slots[start[b]] >= 0 else 0
                         for b, n in enumerate(new)])
        done = (rng.random(6) < 0.2).astype(np.int64)
        ln, free, n_free, kc, vc, err = R.commit(sh, 30, N, start, None, keep, done, slots, ln, table,
                                                 free, left, None, None, kc, vc)
        assert err == 0
        own = _owned(sh, table, ln)
        stack = free[:n_free].tolist()
        assert sorted(own + stack) == list(range(16))
    assert seen == R.NO_PAGES  # the pool did run short

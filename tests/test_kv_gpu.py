"""The paged key/value cache calls and the attention over it, on the GPU,
against the plain 64-bit implementations."""
import dataclasses

import numpy as np
import pytest
import torch

import kv_ref as R
from speculative_decode_verify_gdn_amd import binding as gb

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    gb.lib()


def same(got, want, what):
    np.testing.assert_array_equal(got, want, err_msg=what)


def check_reserve(bt):
    bt.g_reserve()
    table, slots, left, err = bt.r_reserve()
    same(R.host(bt.d["slots"]), slots, "slots")
    same(R.host(bt.d["table"]), table, "block table")
    assert int(bt.d["n_left"]) == left and int(bt.d["err"]) == err
    return table, slots, left


def close(got, want, tol, what=""):
    with np.errstate(invalid="ignore"):
        bad = ~(np.abs(got - want) <= tol)
    bad &= ~(np.isnan(got) & np.isnan(want)) & ~(got == want)
    if bad.any():
        i = tuple(int(x) for x in np.argwhere(bad)[0])
        raise AssertionError("%s: %d of %d outside, first %s: %r, %r +- %r" % (
            what, bad.sum(), bad.size, i, got[i], want[i], tol[i]))


def check_attention(bt, scale=None):
    """Reserve, append, attend; every output against the plain form."""
    table, slots, _ = check_reserve(bt)
    bt.g_append()
    kc, vc, err = bt.r_append(slots)
    same(R.hostf(bt.d["kc"]), kc, "k cache")
    same(R.hostf(bt.d["vc"]), vc, "v cache")
    bt.g_attend(scale=scale)
    want, tol = bt.r_attend(table, kc, vc, scale)
    close(R.hostf(bt.d["o"]).astype(np.float64), want, tol, "o")
    assert int(bt.d["err"]) == 0


# ---- reserve

@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
def test_reserve_lengths_around_pages(page):
    ctx = [0, 0, 1, page - 1, page, page + 1, 3 * page - 2, 5, 0]
    new = [0, 1, page, 1, 1, 0, 2, 2 * page + 3, page]
    check_reserve(R.Batch(1, ctx, new, page=page, pad=5))


def test_reserve_uniform_and_rows_behind():
    check_reserve(R.Batch(2, [3, 20, 0, 64], [7] * 4, packed=False, pad=9))


@pytest.mark.parametrize("B", [1, 255, 256, 257, 700])
def test_reserve_many_sequences(B):
    rng = np.random.default_rng(B)
    check_reserve(R.Batch(B, rng.integers(0, 100, B).tolist(), rng.integers(0, 40, B).tolist()))


def test_reserve_long_prompt():
    check_reserve(R.Batch(5, [10, 33, 0], [5000, 1, 2049], pad=3))


@pytest.mark.parametrize("free", [0, 1, 2, 5, 300])
def test_reserve_pool_runs_short(free):
    """Sequences are served in order until the pages run out; one that needs
    none always is."""
    rng = np.random.default_rng(7)
    new = rng.integers(0, 40, 300).tolist()
    bt = R.Batch(3, rng.integers(0, 60, 300).tolist(), new)
    bt.n_free = free
    bt.upload()
    check_reserve(bt)


def test_reserve_malformed_lengths():
    """Bad lengths leave the sequence out; the others are served."""
    bt = R.Batch(4, [5, 30, 2, 9, 40], [3, 4, 5, 6, 2], pad=4)
    bt.seq_len[1], bt.seq_len[3] = -1, bt.sh.max_blocks * 16 - 1
    bt.upload()
    check_reserve(bt)
    bt = R.Batch(4, [5, 30, 2], [3, 4, 5])
    bt.T = 4  # the third sequence has more than T tokens
    bt.upload()
    bt.g_reserve()
    table, slots, left, err = bt.r_reserve()
    same(R.host(bt.d["slots"])[:7], slots[:7], "slots")
    assert int(bt.d["err"]) == err == R.LENGTH and int(bt.d["n_left"]) == left
    for n_free in (-1, 1 << 30):
        bt = R.Batch(4, [5, 30, 2], [3, 4, 15])
        bt.n_free = n_free
        bt.upload()
        check_reserve(bt)


def test_reserve_bad_page_numbers():
    bt = R.Batch(6, [5, 30, 2], [3, 40, 5])
    bt.table[0, 0] = bt.sh.n_pages
    bt.table[2, 0] = -3
    bt.free[bt.n_free - 1] = 1 << 30
    bt.upload()
    check_reserve(bt)


# ---- append

@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("page", [16, 64, 256])
def test_append(dtype, D, page):
    bt = R.Batch(8, [0, 3, 17, 8, 70], [1, 70, 0, 16, 129], L=2, Hq=3, Hkv=3, D=D, page=page,
                 dtype=dtype, pad=3)
    _, slots, _ = check_reserve(bt)
    bt.g_append()
    kc, vc, err = bt.r_append(slots)
    same(R.hostf(bt.d["kc"]), kc, "k cache")
    same(R.hostf(bt.d["vc"]), vc, "v cache")
    assert int(bt.d["err"]) == err == 0


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_append_slots_in_any_order_and_strided_rows(dtype):
    """Slots of no order, skipped and bad ones, k and v slices of one tensor."""
    rng = np.random.default_rng(5)
    bt = R.Batch(9, [0], [200], L=2, Hkv=2, page=16, dtype=dtype)
    slots = rng.permutation(bt.sh.n_pages * 16)[:200].astype(np.int64)
    slots[[3, 64, 65, 199]] = [-1, bt.sh.n_pages * 16, -2, 1 << 30]
    wide = torch.randn(2, 200, 4 * 2 + 2 + 2, 64, device="cuda").to(dtype)
    k, v = wide[:, :, 8:10], wide[:, :, 10:12]
    d = bt.d
    d["slots"].copy_(torch.tensor(slots))
    gb.kv_append(bt.sh, k, v, d["slots"], d["kc"], d["vc"], dev_err=d["err"])
    kc, vc, err = R.append(bt.sh, R.hostf(k), R.hostf(v), slots, bt.kc, bt.vc)
    same(R.hostf(d["kc"]), kc, "k cache")
    same(R.hostf(d["vc"]), vc, "v cache")
    assert int(d["err"]) == err == R.PAGE


# ---- attention

SHAPES = [  # (Hq, Hkv, D)
    (1, 1, 64), (4, 2, 64), (6, 2, 64), (8, 1, 128), (32, 4, 128), (5, 5, 128), (16, 2, 256),
    (7, 1, 256), (20, 1, 128), (70, 1, 64)]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("Hq,Hkv,D", SHAPES)
def test_attention_single_tokens(Hq, Hkv, D, dtype):
    check_attention(R.Batch(20 + D, [0, 1, 15, 16, 17, 31, 32, 33, 63, 64, 300], [1] * 11, Hq=Hq,
                            Hkv=Hkv, D=D, dtype=dtype, packed=False))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("Hq,Hkv,D", SHAPES)
def test_attention_drafts(Hq, Hkv, D, dtype):
    check_attention(R.Batch(30 + D, [0, 5, 90, 31, 129, 64], [9, 1, 0, 12, 8, 5], Hq=Hq, Hkv=Hkv, D=D,
                            dtype=dtype, pad=4, page=32, garbage=float("nan")))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("T", [1, 2, 7, 16, 33, 63, 64])
def test_attention_trees(T, dtype):
    check_attention(R.Batch(40 + T, [0, 3, 130], [T, max(T - 3, 1), T], Hq=8, Hkv=2, D=128,
                            dtype=dtype, tree=True, pad=1, page=16, garbage=float("nan")))


@pytest.mark.parametrize("Hq,Hkv,D", [(16, 2, 256), (6, 2, 64), (32, 4, 128)])
def test_attention_trees_by_heads(Hq, Hkv, D):
    check_attention(R.Batch(45, [77, 200], [64, 40], Hq=Hq, Hkv=Hkv, D=D, tree=True, page=64))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("Hq,Hkv,D", [(1, 1, 64), (8, 1, 128), (6, 2, 64), (4, 2, 256), (7, 1, 128)])
def test_attention_prompts(Hq, Hkv, D, dtype):
    """Prompts of odd lengths, one behind a cached prefix, one of one token."""
    check_attention(R.Batch(50 + D, [0, 37, 100, 0], [131, 200, 1, 64], Hq=Hq, Hkv=Hkv, D=D,
                            dtype=dtype, pad=2, page=64, garbage=float("inf")))


@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
def test_attention_pages(page):
    check_attention(R.Batch(60, [page - 1, page, 3 * page + 5], [4, 1, 30], page=page, Hq=4, Hkv=1))


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_attention_long_context_split(dtype):
    """One sequence long enough that many workgroups share a row, beside short ones."""
    check_attention(R.Batch(70, [9000, 3, 0, 700], [2, 1, 3, 1], Hq=4, Hkv=1, D=64, dtype=dtype,
                            qmul=3.0))


def test_attention_layers_at_once():
    check_attention(R.Batch(71, [40, 300], [9, 3], L=3, Hq=4, Hkv=2, D=128))


@pytest.mark.parametrize("scale", [0.0, -0.2, 3.0])
def test_attention_scales(scale):
    check_attention(R.Batch(72, [100, 5], [5, 40], Hq=4, Hkv=2, dtype=F32), scale=scale)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("T", [5, 80])
def test_attention_scores_of_great_range(dtype, T):
    """Scores from -2000 to 2000: maxima that rise late, sums that fall away."""
    bt = R.Batch(73, [500, 70], [T, T], Hq=4, Hkv=2, D=64, dtype=dtype, qmul=500.0)
    check_attention(bt)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("tree,T", [(False, 6), (True, 13), (False, 150)])
def test_attention_masked_tokens_hold_nan_and_infinities(tree, T, dtype):
    """A new token whose key or value is not finite changes only the rows that
    attend to it; those follow IEEE arithmetic."""
    bt = R.Batch(74, [45, 3], [T, T], Hq=4, Hkv=2, D=64, dtype=dtype, tree=tree)
    a, c = bt.q_start[0] + T - 2, bt.q_start[1] + T // 2
    bt.v[:, a, :, 5] = np.inf
    bt.v[:, a, :, 6] = -np.inf
    bt.v[:, a, :, 7] = np.nan
    bt.k[:, c, 0, 3] = np.nan
    bt.v[:, c, 0, 9] = np.inf
    bt.upload()
    table, slots, _ = check_reserve(bt)
    bt.g_append()
    kc, vc, _ = bt.r_append(slots)
    bt.g_attend()
    with np.errstate(all="ignore"):
        want, tol = bt.r_attend(table, kc, vc)
    got = R.hostf(bt.d["o"]).astype(np.float64)
    tol = np.where(np.isfinite(want), tol, 0.0)
    close(got, want, tol, "o")
    assert np.isnan(want).any() and np.isinf(want).any() and np.isfinite(want).any()


@pytest.mark.parametrize("Hq,T", [(8, 1), (16, 2), (16, 4), (32, 4), (2, 8), (4, 32), (2, 64)])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_attention_probabilities_of_16_bits_lose_nothing(D, Hq, T):
    """bf16 with at most 64 query rows to a key head: a probability is held to 2^-16
    for the product with V, so that beside fp32's own errors only the output's rounding
    counts.  tol: fp32's, then 2^-16 of sum p |v|, which is at most the largest |v|,
    then 2^-8 of the result as it stands before the last rounding."""
    bt = R.Batch(108, [9, 300, 2000], [T, T, max(1, T - 1)], Hq=Hq, Hkv=2, D=D, page=64)
    table, slots, _ = check_reserve(bt)
    bt.g_append()
    kc, vc, _ = bt.r_append(slots)
    bt.g_attend()
    bt.sh = dataclasses.replace(bt.sh, dtype=F32)  # of the plain form: its tolerance in fp32
    want, tol = bt.r_attend(table, kc, vc)
    tol = tol + 2.0 ** -16 * np.abs(vc).max()
    close(R.hostf(bt.d["o"]).astype(np.float64), want, tol + 2.0 ** -8 * (np.abs(want) + tol), "o")


def test_attention_strided_q():
    bt = R.Batch(75, [50, 9], [3, 20], L=2, Hq=4, Hkv=2, D=64)
    table, slots, _ = check_reserve(bt)
    bt.g_append()
    kc, vc, _ = bt.r_append(slots)
    wide = torch.full((2, bt.N, 4 + 5, 64), float("nan"), device="cuda", dtype=BF16)
    wide[:, :, 2:6] = bt.d["q"]
    bt.d["q"] = wide[:, :, 2:6]
    bt.g_attend()
    want, tol = bt.r_attend(table, kc, vc)
    close(R.hostf(bt.d["o"]).astype(np.float64), want, tol, "o")


@pytest.mark.parametrize("T", [4, 30])
def test_attention_malformed_tree(T):
    """The sequence with the bad parent keeps its rows; the others are right."""
    bt = R.Batch(76, [20, 70, 3], [T, T, T], tree=True, Hq=8, Hkv=2, D=128)
    bt.parent[bt.q_start[1] + 2] = 2
    bt.upload()
    table, slots, _ = check_reserve(bt)
    bt.g_append()
    kc, vc, _ = bt.r_append(slots)
    bt.g_attend()
    bt.parent[bt.q_start[1] + 2] = 0
    want, tol = bt.r_attend(table, kc, vc)
    a, c = bt.q_start[1], bt.q_start[2]
    want[:, a:c], tol[:, a:c] = 3.0, 0.0
    close(R.hostf(bt.d["o"]).astype(np.float64), want, tol, "o")
    assert int(bt.d["err"]) == gb.DEV_ERR_PARENT


@pytest.mark.parametrize("T", [2, 90])
def test_attention_bad_page_numbers(T):
    """A page outside the pool is flagged and not read; the other sequences are
    right.  So are lengths that do not fit."""
    bt = R.Batch(77, [120, 70, 30, 8], [T, T, T, T], Hq=8, Hkv=2, D=128)
    table, slots, _ = check_reserve(bt)
    bt.g_append()
    kc, vc, _ = bt.r_append(slots)
    bad = table.copy()
    bad[1, 0], bad[1, 2] = bt.sh.n_pages, -1
    bt.d["table"].copy_(torch.tensor(bad))
    bt.seq_len[3] = -4
    bt.d["seq_len"].copy_(torch.tensor(bt.seq_len))
    bt.g_attend()
    want, tol = bt.r_attend(table, kc, vc)
    got = R.hostf(bt.d["o"]).astype(np.float64)
    a, c = bt.q_start[1], bt.q_start[2]
    got[:, a:c] = want[:, a:c]
    close(got, want, tol, "o")
    assert int(bt.d["err"]) == gb.DEV_ERR_PAGE | gb.DEV_ERR_LENGTH


@pytest.mark.parametrize("B", [64, 65, 130, 300])
@pytest.mark.parametrize("Hq,T", [(4, 3), (16, 3), (16, 9)])
def test_attention_many_sequences(Hq, T, B):
    """More sequences than a wave or a workgroup has lanes, some of no tokens;
    rows of up to 16, 64 and 128 to a key head."""
    rng = np.random.default_rng(B)
    new = rng.integers(0, T + 1, B).tolist()
    new[0], new[-1] = 0, T
    check_attention(R.Batch(90 + B, rng.integers(0, 90, B).tolist(), new, Hq=Hq, Hkv=1, pad=3))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("Hq,T,tree", [(4, 3, False), (8, 7, True), (8, 30, True), (2, 150, False)])
def test_attention_rows_shared_by_many_workgroups(Hq, T, tree, D, dtype):
    """Contexts long enough to be split, for every size of a row tile, between
    sequences that begin and end inside a workgroup's part."""
    check_attention(R.Batch(91, [40, 5000, 0, 2300], [T, T, 1, T], Hq=Hq, Hkv=1, D=D, dtype=dtype,
                            tree=tree, page=64))


@pytest.mark.parametrize("Hq,T,tree", [(4, 3, False), (4, 3, True), (8, 7, True), (8, 40, True),
                                       (2, 150, False)])
def test_attention_split_rows_with_nan_and_infinities(Hq, T, tree):
    bt = R.Batch(92, [4000, 30], [T, T], Hq=Hq, Hkv=1, D=128, tree=tree)
    a, c = bt.q_start[0] + T - 1, bt.q_start[1] + 1
    bt.v[:, a, :, 5], bt.v[:, a, :, 6] = np.inf, np.nan
    bt.k[:, c, 0, 3] = np.nan
    bt.v[:, c, 0, 9] = -np.inf
    bt.upload()
    table, slots, _ = check_reserve(bt)
    bt.g_append()
    kc, vc, _ = bt.r_append(slots)
    bt.g_attend()
    with np.errstate(all="ignore"):
        want, tol = bt.r_attend(table, kc, vc)
    close(R.hostf(bt.d["o"]).astype(np.float64), want, np.where(np.isfinite(want), tol, 0.0), "o")
    assert np.isnan(want).any() and np.isfinite(want).any()


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("T", [2, 12, 100])
def test_attention_keys_whose_scores_are_infinite(T, dtype):
    """Scores of minus infinity count for nothing, also where they come first and
    fill more than a tile; one of plus infinity makes its row NaN."""
    bt = R.Batch(93, [400, 90], [T, T], Hq=8, Hkv=2, D=64, dtype=dtype)
    bt.q[..., 3] = np.abs(bt.q[..., 3]) + 0.5
    for b, n in ((0, 150), (1, 20)):
        for j in range(n):
            bt.kc[:, bt.table[b, j // 16], 0, j % 16, 3] = -np.inf
    bt.kc[:, bt.table[1, 4], 1, 5, 3] = np.inf
    bt.upload()
    table, slots, _ = check_reserve(bt)
    bt.g_append()
    kc, vc, _ = bt.r_append(slots)
    bt.g_attend()
    with np.errstate(all="ignore"):
        want, tol = bt.r_attend(table, kc, vc)
    tol = np.where(np.isfinite(want), tol, 0.0)
    close(R.hostf(bt.d["o"]).astype(np.float64), want, tol, "o")
    assert np.isnan(want[:, bt.q_start[1]:bt.q_start[2], 4:]).all()
    assert np.isfinite(want[:, :, :4]).all()


def check_not_finite(bt, zero):
    """Rows of `zero` [N,Hq], all of whose scores are minus infinity, are 0; elsewhere
    what is finite in the plain form is right and what is not is not."""
    table, slots, _ = check_reserve(bt)
    bt.g_append()
    kc, vc, _ = bt.r_append(slots)
    bt.g_attend()
    with np.errstate(all="ignore"):
        want, tol = bt.r_attend(table, kc, vc)
    got = R.hostf(bt.d["o"]).astype(np.float64)
    assert (got[:, zero] == 0).all()
    assert np.isnan(want[:, zero]).all()
    got, want, tol = got[:, ~zero], want[:, ~zero], tol[:, ~zero]
    fin = np.isfinite(want)
    assert (np.isfinite(got) == fin).all()
    close(got[fin], want[fin], tol[fin], "o")
    assert fin.any()


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("ctx", [0, 70, 700, 5000])
@pytest.mark.parametrize("Hq,T", [(4, 3), (16, 3), (16, 9)])
def test_attention_values_beside_scores_of_minus_infinity(Hq, T, ctx, dtype):
    """The first sequence's cached keys and first two new ones score minus infinity
    for head 0, and some of their values are not finite.  Its first two rows are 0
    there; the others see a key that counts."""
    bt = R.Batch(104, [ctx, 33], [T, T], Hq=Hq, Hkv=2, D=64, dtype=dtype)
    bt.q[..., 3] = np.abs(bt.q[..., 3]) + 0.5
    for j in range(ctx):
        bt.kc[:, bt.table[0, j // 16], 0, j % 16, 3] = -np.inf
    for j, to in ((40, np.inf), (ctx - 1, -np.inf), (ctx // 2, np.nan)):
        if 0 <= j < ctx:
            bt.vc[:, bt.table[0, j // 16], 0, j % 16 // 8, 5 + j % 3, j % 8] = to
    bt.k[:, :2, 0, 3] = -np.inf
    bt.v[:, 0, 0, 9], bt.v[:, 1, 0, 10] = np.inf, np.nan
    bt.upload()
    zero = np.zeros((bt.N, Hq), bool)
    zero[:2, :Hq // 2] = True
    check_not_finite(bt, zero)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("ctx", [700, 5000])
@pytest.mark.parametrize("Hq,T", [(4, 3), (16, 3), (16, 9)])
def test_attention_infinite_values_of_little_weight(Hq, T, ctx, dtype):
    """An infinite value reaches its rows however small its weight, wherever its
    key lies: among the first keys, whose scores are hundreds below the others'."""
    bt = R.Batch(105, [ctx, 33], [T, T], Hq=Hq, Hkv=2, D=64, dtype=dtype)
    bt.q[..., 3] = np.abs(bt.q[..., 3]) + 0.5
    for j in range(ctx // 2):
        bt.kc[:, bt.table[0, j // 16], 0, j % 16, 3] = -8000.0
    for j, to in ((3, np.inf), (40, -np.inf), (ctx // 2 - 1, np.nan)):
        bt.vc[:, bt.table[0, j // 16], 0, j % 16 // 8, 20 + j % 8, j % 8] = to
    bt.upload()
    check_not_finite(bt, np.zeros((bt.N, Hq), bool))


@pytest.mark.parametrize("scale", [0.0, -0.2, 1e-3])
@pytest.mark.parametrize("T", [2, 9, 60])
def test_attention_scales_of_16_bits(T, scale):
    check_attention(R.Batch(94, [100, 5], [T, T], Hq=8, Hkv=2, tree=True), scale=scale)


@pytest.mark.parametrize("T", [3, 9, 60])
def test_attention_layers_of_tiles(T):
    check_attention(R.Batch(95, [40, 300], [T, T - 1], L=5, Hq=8, Hkv=2, D=128))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("T", [1, 6, 20])
@pytest.mark.parametrize("L", [30, 75])
def test_attention_heads_that_do_not_divide_the_workgroups(L, T, dtype):
    """More key heads over the layers than half of the workgroups, and as many as
    leave a few: workgroups end one head and begin the next, or stay without work."""
    check_attention(R.Batch(107, [700, 90], [T, T], L=L, Hq=16, Hkv=4, D=64, dtype=dtype, page=64))


@pytest.mark.parametrize("T", [3, 9, 60])
def test_attention_without_tokens(T):
    """No new tokens at all: nothing is written."""
    bt = R.Batch(96, [40, 0, 300], [0, 0, 0], Hq=8, Hkv=2, D=128, pad=T)
    bt.T = T
    bt.upload()
    check_attention(bt)
    same(R.hostf(bt.d["o"]), np.full_like(bt.o, 3.0), "o")


@pytest.mark.parametrize("T", [3, 9, 60])
def test_attention_malformed_starts(T):
    """Starts that fall, lie outside or span more than T: those sequences are
    left out, the others are right."""
    bt = R.Batch(97, [40, 20, 300, 8], [T, 1, 2, 2], Hq=8, Hkv=2, D=128)
    table, slots, _ = check_reserve(bt)
    bt.g_append()
    kc, vc, _ = bt.r_append(slots)
    for at, to in ((1, T + 9), (1, T + 1), (4, bt.N + 1), (0, -1), (4, bt.q_start[3] - 1)):
        start = bt.q_start.copy()
        start[at] = to
        bt.d["q_start"].copy_(torch.tensor(start))
        bt.d["o"].fill_(3.0)
        bt.d["err"].zero_()
        bt.g_attend()
        want, tol = R.attend(bt.sh, bt.T, bt.N, start, bt.seq_len, table, None, bt.q,
                             bt.sh.D ** -0.5, kc, vc, bt.o)
        close(R.hostf(bt.d["o"]).astype(np.float64), want, tol, "o")
        assert int(bt.d["err"]) == gb.DEV_ERR_LENGTH


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("T", [3, 30])
def test_cache_beyond_32_bits(T, dtype):
    """Pages whose places lie past 2^32 elements and bytes, in both caches."""
    bt = R.Batch(98, [700, 40, 0], [T, T, T], L=2, Hq=8, Hkv=2, D=256, page=256, dtype=dtype,
                 tree=True)
    small, at = bt.sh, 17000  # 256 pages of 256 tokens of 2 heads: 33.5 million elements
    big = gb.KvShape(small.L, small.B, small.Hq, small.Hkv, small.D, small.page,
                     at + small.n_pages, small.max_blocks, dtype)
    d = bt.d
    caches = {}
    for n in ("kc", "vc"):
        caches[n] = torch.empty(getattr(big, {"kc": "k_cache_shape", "vc": "v_cache_shape"}[n]),
                                dtype=dtype, device="cuda")
        caches[n][:, at:] = d[n]
    assert caches["kc"][0].numel() > 2 ** 31 and caches["kc"].numel() > 2 ** 32
    d.update(caches)
    table, slots, left, _ = bt.r_reserve()
    kc, vc, _ = bt.r_append(slots)
    d["table"].add_(at)
    d["free"] = torch.cat([d["free"] + at, d["free"].new_full((at,), -1)])
    bt.sh = big
    bt.g_reserve()
    same(R.host(d["slots"]), slots + at * 256, "slots")
    bt.g_append()
    bt.g_attend()
    bt.sh = small
    want, tol = bt.r_attend(table, kc, vc)
    close(R.hostf(d["o"]).astype(np.float64), want, tol, "o")
    keep, path = tree_paths(bt, np.random.default_rng(1))
    *_, kc, vc, _ = bt.r_commit(keep, path, None, slots, table, bt.free, left, kc, vc)
    bt.sh = big
    bt.g_commit(keep, path)
    same(R.hostf(d["kc"][:, at:]), kc, "k cache")
    same(R.hostf(d["vc"][:, at:]), vc, "v cache")
    assert int(d["err"]) == 0


def test_attention_same_bits_every_time():
    bt = R.Batch(78, [3000, 40, 700], [9, 300, 1], Hq=8, Hkv=2, D=128)
    check_attention(bt)
    first = bt.d["o"].clone()
    for _ in range(5):
        bt.d["o"].fill_(0)
        bt.d["ws"].fill_(0x5a)
        bt.g_attend()
        assert torch.equal(bt.d["o"][:, :bt.q_start[-1]], first[:, :bt.q_start[-1]])


# ---- commit

def tree_paths(bt, rng):
    keep, path = [], np.full((bt.sh.B, bt.T), -1, np.int64)
    for b in range(bt.sh.B):
        s = int(bt.q_start[b])
        n = int(bt.q_start[b + 1]) - s
        v = int(rng.integers(-1, n)) if n else -1
        way = []
        while v >= 0:
            way.insert(0, v)
            v = int(bt.parent[s + v])
        keep.append(len(way))
        path[b, :len(way)] = way
    return np.array(keep), path


def check_commit(bt, keep, path, done, in_place=False, err=0):
    table, slots, left = check_reserve(bt)
    bt.g_append()
    kc, vc, _ = bt.r_append(slots)
    bt.d["err"].zero_()
    bt.g_commit(keep, path, done, in_place=in_place)
    ln, free, top, kc, vc, want_err = bt.r_commit(keep, path, done, slots, table, bt.free, left, kc, vc)
    assert int(bt.d["err"]) == want_err == err
    got = R.host(bt.d["seq_len" if in_place else "len_out"])
    same(got, ln, "lengths")
    same(R.host(bt.d["free"]), free, "stack")
    assert int(bt.d["n_free"]) == top
    same(R.hostf(bt.d["kc"]), kc, "k cache")
    same(R.hostf(bt.d["vc"]), vc, "v cache")


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("B", [1, 9, 300])
def test_commit_chain(B, in_place):
    rng = np.random.default_rng(B)
    ctx, new = rng.integers(0, 90, B), rng.integers(0, 50, B)
    bt = R.Batch(80, ctx.tolist(), new.tolist(), pad=2)
    keep = np.array([rng.integers(0, n + 1) for n in new])
    check_commit(bt, keep, None, (rng.random(B) < 0.2).astype(np.int64), in_place)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("T", [1, 8, 64])
def test_commit_tree(T, D, dtype):
    rng = np.random.default_rng(T)
    new = [T, max(1, T - 1), T, max(1, T // 2), 0, T]
    bt = R.Batch(81, [0, 5, 15, 16, 40, 100], new, L=2, Hq=3, Hkv=3, D=D, dtype=dtype, tree=True)
    keep, path = tree_paths(bt, rng)
    check_commit(bt, keep, path, np.array([0, 0, 0, 1, 0, 0]))


def test_commit_chain_shaped_long_paths_and_repeats():
    """Paths that skip nodes, go backwards and repeat one: only copies."""
    bt = R.Batch(82, [7, 30], [64, 64], L=1, Hq=2, Hkv=2)
    path = np.stack([np.arange(63, -1, -1), np.full(64, 5)]).astype(np.int64)
    check_commit(bt, np.array([64, 40]), path, None)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_commit_writes_every_kept_row(dtype):
    """Kept rows come from k and v, also those whose place is their own, whatever
    the cache holds there."""
    bt = R.Batch(85, [7, 30], [9, 12], L=2, Hq=4, Hkv=4, D=128, dtype=dtype)
    table, slots, left = check_reserve(bt)
    path = np.full((2, 12), -1, np.int64)
    path[0, :4], path[1, :3] = [0, 1, 5, 8], [0, 2, 3]
    keep = np.array([4, 3])
    bt.g_commit(keep, path, None)
    _, _, _, kc, vc, err = bt.r_commit(keep, path, None, slots, table, bt.free, left, bt.kc, bt.vc)
    assert int(bt.d["err"]) == err == 0
    same(R.hostf(bt.d["kc"]), kc, "k cache")
    same(R.hostf(bt.d["vc"]), vc, "v cache")


def test_commit_gives_back_many_pages():
    """Sequences that end with thousands of pages beside some of a few and none."""
    rng = np.random.default_rng(86)
    ctx = rng.integers(0, 200, 150)
    ctx[[3, 64, 65, 149]] = [40000, 5000, 1, 17000]
    bt = R.Batch(86, ctx.tolist(), rng.integers(0, 40, 150).tolist(), Hq=1, Hkv=1)
    table, slots, left = check_reserve(bt)
    keep = np.array([rng.integers(0, n + 1) for n in np.diff(bt.q_start)])
    done = (rng.random(150) < 0.5).astype(np.int64)
    done[[3, 64, 149]] = 1
    bt.g_commit(keep, None, done)
    out, free, top, *_ = bt.r_commit(keep, None, done, slots, table, bt.free, left, bt.kc, bt.vc)
    same(R.host(bt.d["len_out"]), out, "lengths")
    same(R.host(bt.d["free"])[:top], free[:top], "stack")
    assert int(bt.d["n_free"]) == top and int(bt.d["err"]) == 0


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_commit_from_slices(dtype):
    """k and v are slices of one projection's output."""
    bt = R.Batch(87, [20, 3, 50], [9, 30, 1], L=2, Hq=2, Hkv=2, D=64, dtype=dtype, tree=True)
    table, slots, left = check_reserve(bt)
    wide = torch.full((2, bt.N, 3 + 2 + 2, 64), float("nan"), device="cuda", dtype=dtype)
    wide[:, :, 3:5], wide[:, :, 5:7] = bt.d["k"], bt.d["v"]
    bt.d["k"], bt.d["v"] = wide[:, :, 3:5], wide[:, :, 5:7]
    bt.g_append()
    kc, vc, _ = bt.r_append(slots)
    keep, path = tree_paths(bt, np.random.default_rng(2))
    bt.g_commit(keep, path)
    *_, kc, vc, err = bt.r_commit(keep, path, None, slots, table, bt.free, left, kc, vc)
    assert int(bt.d["err"]) == err == 0
    same(R.hostf(bt.d["kc"]), kc, "k cache")
    same(R.hostf(bt.d["vc"]), vc, "v cache")


def test_commit_errors():
    bt = R.Batch(83, [7, 30, 2, 9], [10, 20, 5, 4])
    path = np.tile(np.arange(20), (4, 1)).astype(np.int64)
    path[2, 1] = 5
    check_commit(bt, np.array([11, 20, 3, -1]), path, None,
                 err=gb.DEV_ERR_N_KEEP | gb.DEV_ERR_PATH)


def test_commit_of_sequences_that_were_not_served():
    """Only the first sequence got pages.  The others keep and give back
    nothing, but the last ends and gives back what it held before."""
    bt = R.Batch(84, [7, 30, 2, 9], [30, 40, 25, 50])
    bt.n_free = 4
    bt.upload()
    slots = bt.r_reserve()[1]
    assert (slots[bt.q_start[:-1]] < 0).tolist() == [False, True, True, True]
    check_commit(bt, np.array([3, 0, 1, 0]), None, np.array([0, 0, 0, 1]), err=R.NO_PAGES)


def test_commit_keeps_nothing_behind_a_first_slot_of_none():
    """A bad page number under the first new token, good ones under the next: the
    counts keep nothing, and so do the caches."""
    bt = R.Batch(106, [13, 30], [9, 12], L=2, Hq=2, Hkv=2)
    bt.table[0, 0] = bt.sh.n_pages
    bt.upload()
    slots = bt.r_reserve()[1]
    assert (slots[:9] >= 0).tolist() == [False] * 3 + [True] * 6
    path = np.stack([np.arange(11, -1, -1) % 9, np.arange(12)]).astype(np.int64)
    check_commit(bt, np.array([8, 5]), path, None, err=R.NO_PAGES)


# ---- together, as a round makes them

def run_rounds(rounds, tree, seed, stream=None, graph=False):
    """Rounds of reserve, append, attend, accept and commit with all lengths on
    the device; checks every step against the plain twins that follow along."""
    rng = np.random.default_rng(seed)
    B, T, V = 3, 6, 50
    bt = R.Batch(seed, [0, 14, 33], [T] * B, Hq=4, Hkv=2, D=64, packed=False, spare=40,
                 extra_blocks=8)
    bt.parent = None
    d, i32 = bt.d, dict(dtype=torch.int32, device="cuda")
    n_keep, bonus = torch.zeros(B, **i32), torch.zeros(B, **i32)
    path = torch.full((B, T), -1, **i32)
    wsp = torch.empty(gb.spec_accept_workspace_bytes(B, T, V), dtype=torch.uint8, device="cuda")
    draft, logits = torch.zeros((B, T), **i32), torch.zeros((B, T + 1, V), device="cuda")
    parent = torch.zeros((B, T), **i32) if tree else None
    d["parent"] = None if parent is None else parent.view(-1)
    done = torch.zeros(B, **i32)

    def call(st):
        bt.g_reserve(st)
        bt.g_append(st)
        bt.g_attend(st)
        gb.spec_accept_prefix(draft, logits, n_keep, path, bonus, wsp, parent=parent,
                              dev_err=d["err"], stream=st)
        bt.g_commit(n_keep, path if tree else None, done, stream=st, in_place=True)

    g = None
    for r in range(rounds):
        for n in ("k", "v", "q"):
            x = torch.randn(d[n].shape, generator=torch.Generator().manual_seed(100 * r + len(n) + ord(n)))
            setattr(bt, n, x.to(BF16).float().numpy())
            d[n].copy_(x)
        dr = rng.integers(0, 4, (B, T))
        lg = rng.standard_normal((B, T + 1, V)).astype(np.float32)
        for b in range(B):
            for t in range(T + 1):
                lg[b, t, rng.integers(0, 4)] += 9.0
        draft.copy_(torch.tensor(dr))
        logits.copy_(torch.tensor(lg))
        par = None
        if tree:
            par = np.array([R.random_tree(rng, T) for _ in range(B)])
            parent.copy_(torch.tensor(par))
            bt.parent = par.reshape(-1)
        dn = (rng.random(B) < 0.15).astype(np.int64)
        done.copy_(torch.tensor(dn))
        torch.cuda.synchronize()
        if not graph:
            call(stream)
        else:
            if g is None:
                st = torch.cuda.Stream()
                g = torch.cuda.CUDAGraph()
                with torch.cuda.stream(st):
                    with torch.cuda.graph(g, stream=st):
                        call(st)
                torch.cuda.synchronize()
            (torch.randn(1 << 14, device="cuda") * 2).sum().item()
            g.replay()
        torch.cuda.synchronize()
        assert int(d["err"]) == 0
        table, slots, left, err = bt.r_reserve()
        assert err == 0
        bt.kc, bt.vc, _ = bt.r_append(slots)
        want, tol = bt.r_attend(table, bt.kc, bt.vc)
        close(R.hostf(d["o"]).astype(np.float64), want, tol, "o of round %d" % r)
        nk, pth = R.host(n_keep), R.host(path)
        ln, free, top, bt.kc, bt.vc, err = bt.r_commit(nk, pth if tree else None, dn, slots, table,
                                                       bt.free, left, bt.kc, bt.vc)
        assert err == 0
        bt.table, bt.seq_len, bt.free, bt.n_free = table, ln, free, top
        same(R.host(d["seq_len"]), ln, "lengths")
        same(R.host(d["free"]), free, "stack")
        same(R.hostf(d["kc"]), bt.kc, "k cache")
        same(R.hostf(d["vc"]), bt.vc, "v cache")
        assert int(d["n_free"]) == top
    assert bt.seq_len.max() > 0


@pytest.mark.parametrize("graph", [False, True])
@pytest.mark.parametrize("tree", [False, True])
def test_rounds_together(tree, graph):
    run_rounds(7, tree, 90 + tree, graph=graph)


def test_calls_follow_the_current_stream():
    """Without a stream argument a call goes to the current one: here behind work
    that gives it its inputs."""
    bt, want = (R.Batch(93, [2000, 5], [3, 20], Hq=8, Hkv=2, D=128) for _ in range(2))
    want.g_reserve(), want.g_append(), want.g_attend()
    q = bt.d["q"].clone()
    bt.d["q"].zero_()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        x = torch.randn(4096, 4096, device="cuda")
        for _ in range(20):
            x = x @ x * 1e-3
        bt.d["q"].copy_(q)
        bt.g_reserve(), bt.g_append(), bt.g_attend()
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(bt.d["o"], want.d["o"])


def test_two_streams_at_once():
    """Two batches on two streams with no wait between them end where they end
    alone."""
    def make(seed):
        return R.Batch(seed, [2000, 5, 90], [3, 200, 1], Hq=8, Hkv=2, D=128)

    alone = [make(91), make(92)]
    for bt in alone:
        bt.g_reserve(), bt.g_append(), bt.g_attend()
    both, streams = [make(91), make(92)], [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(3):
        for bt, st in zip(both, streams):
            bt.g_reserve(st), bt.g_append(st), bt.g_attend(st)
    torch.cuda.synchronize()
    for a, b in zip(alone, both):
        for n in ("slots", "table", "kc", "vc", "o", "n_left"):
            assert torch.equal(a.d[n], b.d[n]), n


# ---- rows of no sequence

STARTS = [  # of sequences of 3, 4, 5 and 2 tokens, T = 5, 18 rows: which start, and its value
    {2: 12}, {3: 14}, {2: 1}, {0: -1}, {0: 2}, {0: 17}, {4: 19}, {4: 11}, {4: 3}, {4: -1},
    {1: 1 << 30}, {1: -(1 << 31)}, {0: 5, 1: 4, 2: 3, 3: 2, 4: 1}, {0: 18, 1: 0, 2: 18, 3: 0, 4: 18}]


@pytest.mark.parametrize("at", STARTS, ids=str)
def test_reserve_clears_rows_of_no_sequence(at):
    """Whatever the starts, every row that no served sequence owns gets slot -1,
    and no other row does: kv_append runs on the same array and writes where it says."""
    bt = R.Batch(101, [5, 30, 2, 40], [3, 4, 5, 2], Hkv=1, Hq=1, pad=4)
    for i, v in at.items():
        bt.q_start[i] = v
    bt.upload()
    bt.d["slots"].copy_(torch.arange(bt.N) * 3 % (bt.sh.n_pages * 16))  # an earlier round's
    _, slots, _ = check_reserve(bt)
    bt.g_append()
    kc, vc, _ = bt.r_append(slots)
    same(R.hostf(bt.d["kc"]), kc, "k cache")
    same(R.hostf(bt.d["vc"]), vc, "v cache")


@pytest.mark.parametrize("T", [4, 39])
@pytest.mark.parametrize("B", [3, 256, 700])
def test_reserve_clears_rows_of_sequences_too_long(B, T):
    rng = np.random.default_rng(B)
    bt = R.Batch(102, rng.integers(0, 100, B).tolist(), rng.integers(0, 40, B).tolist(), pad=5)
    bt.T = T
    bt.seq_len[B // 2] = -1
    bt.upload()
    bt.d["slots"].fill_(16)
    check_reserve(bt)


def test_reserve_clears_many_rows():
    """More rows than are looked at in one go, of a sequence too long between two
    that are served."""
    bt = R.Batch(103, [3, 900, 70], [70000, 75000, 60000], Hkv=1, Hq=1, page=256, pad=70000)
    bt.T = 70000
    bt.upload()
    bt.d["slots"].fill_(16)
    check_reserve(bt)

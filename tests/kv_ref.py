"""Plain 64-bit implementations of the paged cache calls and the attention over
it, on host arrays, and the device-side set-up that their tests share.  Loops
over sequences, tokens and heads, straight from the definitions."""
from __future__ import annotations

import numpy as np
import torch

from speculative_decode_verify_gdn_amd import binding as gb

LENGTH, PAGE, NO_PAGES = gb.DEV_ERR_LENGTH, gb.DEV_ERR_PAGE, gb.DEV_ERR_NO_PAGES


def up(a, b):
    return -(-a // b)


def spans(B, T, N, q_start, seq_len, room):
    """(first row, new tokens, cached tokens, well formed) of each sequence."""
    out = []
    for b in range(B):
        s, e = (b * T, b * T + T) if q_start is None else (q_start[b], q_start[b + 1])
        ok = 0 <= s <= e <= N and e - s <= T
        rows = e - s if ok else 0
        c = seq_len[b]
        ok2 = ok and c >= 0 and c + rows <= room
        out.append((s, rows, c, ok2))
    return out


def reserve(sh, T, N, q_start, seq_len, table, free, n_free):
    """(block table, slots, pages left, error bits)."""
    table, err, page = table.copy(), 0, sh.page
    sp = spans(sh.B, T, N, q_start, seq_len, sh.max_blocks * page)
    slots = np.full(N, -1, np.int64)
    if not 0 <= n_free <= sh.n_pages:
        err, n_free = err | NO_PAGES, 0
    upto, top = 0, n_free
    for b, (s, n, c, ok) in enumerate(sp):
        if not ok:
            err |= LENGTH
            continue
        have, want = up(c, page), up(c + n, page)
        upto += want - have
        if want > have and upto > n_free:
            err |= NO_PAGES
            continue
        for j in range(have, want):
            top -= 1
            pg = free[top]
            if not 0 <= pg < sh.n_pages:
                err, pg = err | PAGE, -1
            table[b, j] = pg
        for i in range(n):
            pg = table[b, (c + i) // page]
            if 0 <= pg < sh.n_pages:
                slots[s + i] = pg * page + (c + i) % page
            else:
                err |= PAGE
    return table, slots, top, err


def place(sh, slot):
    return slot // sh.page, slot % sh.page


def append(sh, k, v, slots, kc, vc):
    """New caches and error bits."""
    kc, vc, err = kc.copy(), vc.copy(), 0
    for t, s in enumerate(slots):
        if s == -1:
            continue
        if not 0 <= s < sh.n_pages * sh.page:
            err |= PAGE
            continue
        pg, off = place(sh, s)
        kc[:, pg, :, off] = k[:, t]
        vc[:, pg, :, off // 8, :, off % 8] = v[:, t]
    return kc, vc, err


def commit(sh, T, N, q_start, path, n_keep, done, slots, seq_len, table, free, n_left, k, v, kc, vc):
    """(lengths, stack, pages free, k cache, v cache, error bits)."""
    free, kc, vc, err, page = free.copy(), kc.copy(), vc.copy(), 0, sh.page
    out, top = seq_len.copy(), n_left
    for b, (s, n, c, ok) in enumerate(spans(sh.B, T, N, q_start, seq_len, sh.max_blocks * page)):
        if not ok:
            err |= LENGTH
            continue
        keep, served = n_keep[b], True
        if not 0 <= keep <= n:
            err, keep = err | gb.DEV_ERR_N_KEEP, 0
        if n > 0 and slots[s] < 0:
            served = False
            err |= NO_PAGES if keep > 0 else 0
            keep = 0
        if path is not None and any(not 0 <= path[b, i] < n for i in range(keep)):
            err, keep = err | gb.DEV_ERR_PATH, 0
        if path is not None:
            for i in range(keep):
                if slots[s + i] >= 0:
                    pg, off = place(sh, slots[s + i])
                    kc[:, pg, :, off] = k[:, s + path[b, i]]
                    vc[:, pg, :, off // 8, :, off % 8] = v[:, s + path[b, i]]
        ln = 0 if done is not None and done[b] else c + keep
        for j in range(up(ln, page), up(c + n if served else c, page)):
            free[top] = table[b, j]
            top += 1
        out[b] = ln
    return out, free, top, kc, vc, err


def attend(sh, T, N, q_start, seq_len, table, parent, q, scale, kc, vc, o):
    """New o in 64 bits (rows of no sequence keep o's values), and how far a
    kernel with fp32 sums may be off, element by element.

    With A = sum_j p_j |v_j|, n keys and Z = max_j |scale| sum_d |q_d k_jd|:
      a score is a sum of D products in fp32, off by at most (D + 2) 2^-24 Z,
      scaled into base 2 and reduced by the maximum (three more roundings of
      numbers up to 2 Z); its exponential takes that as a relative error, plus
      2^-22 for exp2 itself.  It enters p above and below the fraction bar;
      sums over n keys add at most n 2^-24 each, above and below, and as much
      again covers the rescalings by the running maximum;
      bf16 rounds each probability once (2^-8 of it) and the output once.
    """
    o = o.astype(np.float64).copy()
    tol = np.zeros_like(o)
    bf16 = sh.dtype == torch.bfloat16
    G = sh.Hq // sh.Hkv
    for b, (s, n, c, ok) in enumerate(spans(sh.B, T, N, q_start, seq_len, sh.max_blocks * sh.page)):
        if not ok or n == 0:
            continue
        j = np.arange(c + n)
        pg, off = table[b, j // sh.page], j % sh.page
        live = np.zeros((n, c + n), bool)
        live[:, :c] = True
        for i in range(n):
            if parent is None:
                live[i, c:c + i + 1] = True
            else:
                u = i
                while u >= 0:
                    live[i, c + u] = True
                    u = parent[s + u]
        for l in range(sh.L):
            for h in range(sh.Hkv):
                K = kc[l, pg, h, off].astype(np.float64)
                V = vc[l, pg, h, off // 8, :, off % 8].astype(np.float64)
                aK, aV = np.abs(K), np.abs(V)
                for i in range(n):
                    w = live[i] if parent is not None else slice(0, c + i + 1)
                    Q = q[l, s + i, h * G:(h + 1) * G].astype(np.float64)
                    z = scale * (Q @ K[w].T)
                    p = np.exp(z - z.max(-1, keepdims=True))
                    p /= p.sum(-1, keepdims=True)
                    res = p @ V[w]
                    Z = abs(scale) * (np.abs(Q) @ aK[w].T)
                    Z = Z[np.isfinite(Z)].max(initial=0.0)  # scores of -inf count for nothing
                    rel = 2 * ((sh.D + 2 + 6) * 2.0 ** -24 * Z + 2.0 ** -22) + 4 * p.shape[1] * 2.0 ** -24
                    A = p @ aV[w]
                    t = A * (rel + (2.0 ** -8 if bf16 else 0.0))
                    o[l, s + i, h * G:(h + 1) * G] = res
                    tol[l, s + i, h * G:(h + 1) * G] = t + (2.0 ** -8 if bf16 else 2.0 ** -24) * (np.abs(res) + t)
    return o, tol


def random_tree(rng, n, depth=8):
    par, dep = [], []
    for v in range(n):
        opts = [-1] + [u for u in range(v) if dep[u] < depth - 1]
        p = int(opts[rng.integers(len(opts))])
        par.append(p)
        dep.append(0 if p < 0 else dep[p] + 1)
    return par


class Batch:
    """A page pool with sequences of given lengths, and a round's new tokens:
    host arrays, and their device twins under the same names in `d`."""

    def __init__(self, seed, ctx, new, *, L=1, Hq=4, Hkv=2, D=64, page=16, dtype=torch.bfloat16,
                 packed=True, pad=0, spare=3, tree=False, extra_blocks=1, device="cuda", qmul=1.0,
                 garbage=None):
        rng = np.random.default_rng(seed)
        B = len(ctx)
        self.T = max(max(new), 1)
        start = np.concatenate([[0], np.cumsum(new)]).astype(np.int64)
        assert packed or all(n == self.T for n in new)
        self.N = max(1, int(start[-1]) + pad)
        self.q_start = start if packed else None
        self.seq_len = np.array(ctx, dtype=np.int64)
        have = [up(c, page) for c in ctx]
        want = [up(c + n, page) for c, n in zip(ctx, new)]
        n_pages = sum(want) + spare
        self.sh = gb.KvShape(L, B, Hq, Hkv, D, page, n_pages, max(max(want), 1) + extra_blocks, dtype)
        ids = rng.permutation(n_pages)
        self.table = np.full((B, self.sh.max_blocks), -1, np.int64)
        at = 0
        for b in range(B):
            self.table[b, :have[b]] = ids[at:at + have[b]]
            at += have[b]
        self.free = np.concatenate([ids[at:], ids[:at]]).astype(np.int64)
        self.n_free = n_pages - at

        def draw(*shape, mul=1.0):
            x = torch.from_numpy(rng.standard_normal(shape, dtype=np.float32) * np.float32(mul))
            return x.to(dtype).float().numpy()

        self.k, self.v = draw(L, self.N, Hkv, D), draw(L, self.N, Hkv, D)
        self.q = draw(L, self.N, Hq, D, mul=qmul)
        self.kc, self.vc = draw(*self.sh.k_cache_shape), draw(*self.sh.v_cache_shape)
        self.parent = None
        if tree:
            self.parent = np.array(sum([random_tree(rng, n) for n in new], []) + [7] * pad, np.int64)
        self.o = np.full((L, self.N, Hq, D), 3.0, np.float32)
        if garbage is not None:  # places that hold no cached token
            keep_k = np.zeros(self.kc.shape, bool)
            keep_v = np.zeros(self.vc.shape, bool)
            for b in range(B):
                for j in range(ctx[b]):
                    pg, off = self.table[b, j // page], j % page
                    keep_k[:, pg, :, off] = True
                    keep_v[:, pg, :, off // 8, :, off % 8] = True
            self.kc[~keep_k] = garbage
            self.vc[~keep_v] = garbage
        self.device = device
        self.d = {}
        if device is not None:
            self.upload()

    def upload(self):
        i32 = dict(dtype=torch.int32, device=self.device)
        fl = dict(dtype=self.sh.dtype, device=self.device)
        for n in ("q_start", "seq_len", "table", "free", "parent"):
            x = getattr(self, n)
            self.d[n] = None if x is None else torch.tensor(x, **i32)
        for n in ("k", "v", "q", "kc", "vc", "o"):
            self.d[n] = torch.from_numpy(getattr(self, n)).to(**fl)
        self.d["n_free"] = torch.tensor([self.n_free], **i32)
        self.d["n_left"] = torch.full((1,), -7, **i32)
        self.d["slots"] = torch.full((self.N,), -9, **i32)
        self.d["len_out"] = torch.full((self.sh.B,), -5, **i32)
        self.d["err"] = torch.zeros(1, **i32)
        self.d["ws"] = torch.full((gb.attn_verify_workspace_bytes(self.sh, self.T, self.N),), 0xff,
                                  dtype=torch.uint8, device=self.device)

    # device calls
    def g_reserve(self, stream=None):
        d = self.d
        gb.kv_reserve(self.sh, d["seq_len"], d["table"], d["free"], d["n_free"], d["n_left"],
                      d["slots"], self.T, q_start=d["q_start"], dev_err=d["err"], stream=stream)

    def g_append(self, stream=None):
        d = self.d
        gb.kv_append(self.sh, d["k"], d["v"], d["slots"], d["kc"], d["vc"], dev_err=d["err"],
                     stream=stream)

    def g_attend(self, stream=None, scale=None):
        d = self.d
        gb.attn_verify(self.sh, d["q"], d["seq_len"], d["table"], d["kc"], d["vc"], d["o"], d["ws"],
                       self.T, q_start=d["q_start"], parent=d["parent"], scale=scale,
                       dev_err=d["err"], stream=stream)

    def g_commit(self, n_keep, path=None, done=None, stream=None, in_place=False):
        d = self.d
        i32 = dict(dtype=torch.int32, device=self.device)

        def dev(x):
            return x if x is None or isinstance(x, torch.Tensor) else torch.tensor(x, **i32)

        gb.kv_commit(self.sh, d["k"], d["v"], d["slots"], dev(n_keep), d["seq_len"],
                     d["seq_len"] if in_place else d["len_out"], d["table"], d["free"],
                     d["n_left"], d["n_free"], d["kc"], d["vc"], self.T, q_start=d["q_start"],
                     path=dev(path), done=dev(done), dev_err=d["err"], stream=stream)

    # the plain twins
    def r_reserve(self):
        return reserve(self.sh, self.T, self.N, self.q_start, self.seq_len, self.table, self.free,
                       self.n_free)

    def r_append(self, slots):
        return append(self.sh, self.k, self.v, slots, self.kc, self.vc)

    def r_attend(self, table, kc, vc, scale=None):
        return attend(self.sh, self.T, self.N, self.q_start, self.seq_len, table, self.parent,
                      self.q, self.sh.D ** -0.5 if scale is None else scale, kc, vc, self.o)

    def r_commit(self, n_keep, path, done, slots, table, free, n_left, kc, vc):
        return commit(self.sh, self.T, self.N, self.q_start, path, n_keep, done, slots,
                      self.seq_len, table, free, n_left, self.k, self.v, kc, vc)


def host(t):
    return t.detach().cpu().to(torch.int64).numpy()


def hostf(t):
    return t.detach().cpu().float().numpy()

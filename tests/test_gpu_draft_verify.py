"""The operators together, as a decoder uses them: a prompt's projection, head
norm and rotation into the cache, attention; then a tree of drafted tokens
through the same cache, the logits and the log probabilities that judge the
drafts. Every step is checked against 64 bits on what the step before it left."""
import numpy as np
import pytest
import torch

import mxfp4_routed_expert_sigmoid_amd as k3
import attn_ref as ref

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not torch.cuda.is_available(), reason="no GPU")]
DEV, BF, U8, I32 = "cuda:0", torch.bfloat16, torch.uint8, torch.int32
H, HQ, HKV, D, V, PAGE = 256, 8, 2, 64, 1000, 16
EPS = 1e-5


def _matrix(rows, cols, g):
    w = torch.randint(0, 256, (rows, cols // 2), dtype=U8, device=DEV, generator=g)
    return w, torch.full((rows, cols // 32), 121, dtype=U8, device=DEV)


def _np(t):
    return t.double().cpu().numpy()


class Layer:
    def __init__(self, x8):
        g = torch.Generator(device=DEV).manual_seed(7)
        self.qkv, self.o, self.head = _matrix((HQ + 2 * HKV) * D, H, g), _matrix(H, HQ * D, g), _matrix(V, H, g)
        self.gamma = 1 + 0.1 * torch.randn(H, device=DEV, generator=g)
        self.gq, self.gk = (1 + 0.1 * torch.randn(D, device=DEV, generator=g) for _ in range(2))
        self.freq = torch.tensor([10000.0 ** (-2 * i / D) for i in range(D // 2)], device=DEV)
        self.x8, pages = x8, 24
        kind = U8 if x8 else BF
        self.kc, self.vc = (torch.zeros((pages, HKV, PAGE, D), dtype=kind, device=DEV) for _ in range(2))
        self.ks, self.vs = ((torch.zeros((pages, HKV, PAGE, D // 32), dtype=U8, device=DEV) for _ in range(2))
                            if x8 else (None, None))
        self.pages = torch.randperm(pages, device=DEV, generator=g).to(I32).view(2, 12).contiguous()   # two sequences

    def place(self, b, pos):
        return self.pages[b, pos // PAGE].long() * PAGE + pos % PAGE

    def before(self, h, pos, slots, q, k_out, v_copy):
        """Norm, projection, head norm and rotation: q, and keys and values in the cache (and in k_out, v_copy)."""
        T = h.shape[0]
        x = torch.empty((T, H), dtype=BF, device=DEV)
        k3.add_norm(h, self.gamma, EPS, x=x)
        y = torch.empty((T, (HQ + 2 * HKV) * D), dtype=BF, device=DEV)
        k3.linear(*self.qkv, x, y)
        yq, yk, yv = (y[:, a * D:(a + n) * D].view(T, n, D) for a, n in ((0, HQ), (HQ, HKV), (HQ + HKV, HKV)))
        k3.qk_norm_rope(yq, yk, pos, self.freq, gamma_q=self.gq, gamma_k=self.gk, eps=EPS, q_out=q, k_out=k_out, v=yv,
                        kc=self.kc, vc=self.vc, ks=self.ks, vs=self.vs, slots=slots)
        if v_copy is not None:
            v_copy.copy_(yv)

    def after(self, h, a):
        """The output projection into the stream and the logits of the new stream."""
        T = h.shape[0]
        k3.linear(*self.o, a.view(T, HQ * D), h, accumulate=True)
        x, logits = torch.empty((T, H), dtype=BF, device=DEV), torch.empty((T, V), device=DEV)
        k3.add_norm(h, self.gamma, EPS, x=x)
        k3.linear(*self.head, x, logits)
        return logits

    def cached(self, b, n):
        """The first n keys and values of a sequence as the cache holds them, 64 bits."""
        p = np.arange(n)
        ids = self.pages[b].cpu().numpy()[p // PAGE]
        out = []
        for c, s in ((self.kc, self.ks), (self.vc, self.vs)):
            x = ref.mxfp8_values(c.cpu().numpy(), s.cpu().numpy()) if self.x8 else _np(c)
            out.append(x[ids, :, p % PAGE])
        return out


@pytest.mark.parametrize("x8", [False, True])
def test_prompt_then_drafts(x8):
    L = Layer(x8)
    g = torch.Generator(device=DEV).manual_seed(3)
    lens = [37, 70]
    T = sum(lens)
    h = torch.randn((T, H), device=DEV, generator=g)
    seq = torch.tensor([0] * lens[0] + [1] * lens[1], device=DEV)
    pos = torch.cat([torch.arange(n, device=DEV) for n in lens]).to(I32)
    q, k, v = (torch.empty((T, n, D), dtype=BF, device=DEV) for n in (HQ, HKV, HKV))
    L.before(h, pos, L.place(seq, pos.long()), q, k, v)
    cu = torch.tensor([0, lens[0], T], dtype=I32, device=DEV)
    a, lse = torch.empty_like(q), torch.empty((T, HQ), device=DEV)
    k3.attention(q, k, v, cu, a, lse=lse)
    torch.cuda.synchronize()
    first = 0
    for b, n in enumerate(lens):
        kc, vc = L.cached(b, n)
        if not x8:
            assert np.array_equal(kc, _np(k)[first:first + n]) and np.array_equal(vc, _np(v)[first:first + n])
        for hd in range(HQ):
            r = slice(first, first + n)
            want = ref.attend(_np(q)[r, hd], _np(k)[r, hd // 4], _np(v)[r, hd // 4], np.tri(n, dtype=bool), D ** -0.5)
            ref.check_rows(_np(a)[r, hd], _np(lse)[r, hd], *want, f"prompt {b} head {hd}")
        first += n
    L.after(h, a)

    # trees of drafted tokens: parents by number, -1 the prompt's last token
    parents = [[-1, 0, 0, 1, 2], [-1, -1, 1]]
    ns = [len(p) for p in parents]
    words, depth = [], []
    for p in parents:
        w, d = [], []
        for i, up in enumerate(p):
            w.append((w[up] if up >= 0 else 0) | 1 << i)
            d.append(d[up] + 1 if up >= 0 else 0)
        words += w
        depth += d
    N = sum(ns)
    h = torch.randn((N, H), device=DEV, generator=g)
    seq = torch.tensor([0] * ns[0] + [1] * ns[1], device=DEV)
    ctx = torch.tensor(lens, device=DEV)
    behind = torch.cat([torch.arange(n, device=DEV) for n in ns])
    pos = (ctx[seq] + torch.tensor(depth, device=DEV)).to(I32)             # the rotation goes by depth,
    slots = L.place(seq, ctx[seq] + behind)                               # the place by number
    q = torch.empty((N, HQ, D), dtype=BF, device=DEV)
    L.before(h, pos, slots, q, None, None)
    a, lse = torch.empty_like(q), torch.empty((N, HQ), device=DEV)
    cu = torch.tensor([0, ns[0], N], dtype=I32, device=DEV)
    k3.tree_attention(q, L.kc, L.vc, L.pages, ctx.to(I32), a, ks=L.ks, vs=L.vs, cu_q=cu, max_q=max(ns),
                      tree=torch.tensor(words, device=DEV), lse=lse)
    torch.cuda.synchronize()
    first = 0
    for b, n in enumerate(ns):
        kc, vc = L.cached(b, lens[b] + n)
        see = np.ones((n, lens[b] + n), bool)
        for i in range(n):
            for j in range(n):
                see[i, lens[b] + j] = words[first + i] >> j & 1
        for hd in range(HQ):
            r = slice(first, first + n)
            want = ref.attend(_np(q)[r, hd], kc[:, hd // 4], vc[:, hd // 4], see, D ** -0.5)
            ref.check_rows(_np(a)[r, hd], _np(lse)[r, hd], *want, f"drafts {b} head {hd}")
        first += n
    logits = L.after(h, a)
    # each drafted token's children are judged by its logits
    ids = torch.randint(0, V, (N, 3), device=DEV, generator=g).to(I32)
    lp, ent = torch.empty((N, 3), device=DEV), torch.empty(N, device=DEV)
    top, top_lp = torch.empty((N, 4), dtype=I32, device=DEV), torch.empty((N, 4), device=DEV)
    k3.logprobs(logits, ids=ids, lp=lp, entropy=ent, top_ids=top, top_lp=top_lp)
    x = logits.cpu().numpy()
    for t in range(N):
        want, e, order, best, tol, etol = ref.logprobs(x[t], ids[t].tolist(), 4)
        assert (np.abs(_np(lp)[t] - want) <= tol + ref.U32 * np.abs(want)).all()
        assert abs(float(ent[t]) - e) <= etol and top[t].tolist() == order.tolist()
        assert (np.abs(_np(top_lp)[t] - best) <= tol + ref.U32 * np.abs(best)).all()

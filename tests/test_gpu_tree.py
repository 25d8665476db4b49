"""k3moe_tree_attention against its formula in 64 bits: single tokens, trees and
chains, both kinds of cache, page sizes, lengths around tiles and pages, bad
pages, empty rows, masked infinities, one workspace for several calls."""
import numpy as np
import pytest
import torch

import mxfp4_routed_expert_sigmoid_amd as k3
import attn_ref as ref

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not torch.cuda.is_available(), reason="no GPU")]
DEV = "cuda:0"
BF = torch.bfloat16


class Case:
    """Drafted tokens over a cache whose unused places hold NaN."""

    def __init__(self, lens, ns, Hq, Hkv, D, Dv, page=16, x8=False, words=None, seed=0, sharp=1.0, spare=2, pad=0):
        g = torch.Generator().manual_seed(seed)
        self.lens, self.ns, self.page, self.x8, self.sharp = lens, ns, page, x8, sharp
        self.Hq, self.Hkv, self.D, self.Dv = Hq, Hkv, D, Dv
        need = [-(-(max(a, 0) + n) // page) for a, n in zip(lens, ns)]
        total, width = sum(need) + spare, max(need + [0]) + 1
        order = torch.randperm(total, generator=g).tolist()
        self.table = np.full((len(lens), width), -1, np.int32)
        for b, m in enumerate(need):
            self.table[b, :m] = [order.pop() for _ in range(m)]
        self.k = np.full((total, Hkv, page, D), np.nan)
        self.v = np.full((total, Hkv, page, Dv), np.nan)
        for b, (a, n) in enumerate(zip(lens, ns)):
            p = np.arange(max(a, 0) + n)
            for x in (self.k, self.v):
                x[self.table[b, p // page], :, p % page] = torch.randn((len(p), Hkv, x.shape[3]), generator=g).numpy()
        self.cache = {}
        for name in ("k", "v"):
            x = getattr(self, name)
            if x8:
                hole = np.isnan(x)
                q, s = ref.mxfp8_pool(np.where(hole, 0.0, x))
                q[hole] = 0x7f
                setattr(self, name, ref.mxfp8_values(q, s))
                self.cache[name + "c"], self.cache[name + "s"] = torch.tensor(q, device=DEV), torch.tensor(s, device=DEV)
            else:
                bits = ref.bf16(x)
                setattr(self, name, ref.unbf16(bits))
                self.cache[name + "c"] = torch.tensor(bits.view(np.int16), device=DEV).view(BF)
        T = sum(ns)
        self.T = T
        self.words = words
        self.q = (sharp * torch.randn((T, Hq * D + pad), generator=g)).to(BF).to(DEV)[:, :Hq * D].view(T, Hq, D)
        self.pages = torch.tensor(self.table, device=DEV)
        self.dlens = torch.tensor(lens, dtype=torch.int32, device=DEV)
        self.cu = torch.tensor([0] + list(np.cumsum(ns)), dtype=torch.int32, device=DEV)

    def see(self, b):
        a, n = max(self.lens[b], 0), self.ns[b]
        s = np.zeros((n, a + n), bool)
        s[:, :a] = True
        first = sum(self.ns[:b])
        for i in range(n):
            w = (1 << (i + 1)) - 1 if self.words is None else self.words[first + i]
            for j in range(n):
                s[i, a + j] = w >> j & 1
        pos = np.arange(a + n) // self.page
        ids = np.where(pos < self.table.shape[1], self.table[b, np.minimum(pos, self.table.shape[1] - 1)], -1)
        return s & ((ids >= 0) & (ids < self.k.shape[0]))[None, :]

    def run(self, uniform=False, lse=True, ws=None, out=None, stream=None, max_q=None):
        out = torch.full((self.T, self.Hq, self.Dv), 5.0, dtype=BF, device=DEV) if out is None else out
        l = torch.full((self.T, self.Hq), 5.0, device=DEV) if lse else None
        tree = None
        if self.words is not None:
            tree = torch.tensor([w - (1 << 64) if w >> 63 else w for w in self.words], dtype=torch.int64, device=DEV)
        k3.tree_attention(self.q, pages=self.pages, lens=self.dlens, out=out, cu_q=None if uniform else self.cu,
                          max_q=max_q or max(self.ns + [1]), tree=tree, lse=l, workspace=ws, stream=stream, **self.cache)
        return out, l

    def check(self, out, lse, heads=None, seqs=None):
        torch.cuda.synchronize()
        o, q = out.double().cpu().numpy(), self.q.double().cpu().numpy()
        l = None if lse is None else lse.double().cpu().numpy()
        first = 0
        for b, (a, n) in enumerate(zip(self.lens, self.ns)):
            if seqs is None or b in seqs:
                see = self.see(b)
                p = np.arange(see.shape[1])
                ids = self.table[b, np.minimum(p // self.page, self.table.shape[1] - 1)]
                ids = np.where((ids >= 0) & (ids < self.k.shape[0]), ids, 0)
                for h in heads or range(self.Hq):
                    kv = h // (self.Hq // self.Hkv)
                    want = ref.attend(q[first:first + n, h], self.k[ids, kv, p % self.page], self.v[ids, kv, p % self.page],
                                      see, self.D ** -0.5)
                    ref.check_rows(o[first:first + n, h], None if l is None else l[first:first + n, h], *want,
                                   f"sequence {b} ({a} + {n}) head {h}")
            first += n


def _tree(ns, seed=0):
    rng = np.random.default_rng(seed)
    words = []
    for n in ns:
        w = []
        for i in range(n):
            up = int(rng.integers(-1, i)) if i else -1
            w.append((w[up] if up >= 0 else 0) | 1 << i)
        words += w
    return words


DIMS = [(64, 64), (128, 128), (192, 128)]


@pytest.mark.parametrize("D,Dv", DIMS)
@pytest.mark.parametrize("x8", [False, True])
@pytest.mark.parametrize("lens", [[0], [1, 15, 16], [62, 63, 64, 65], [127, 128, 300], [1000, 3, 0, 517]])
def test_single_tokens(D, Dv, x8, lens):
    c = Case(lens, [1] * len(lens), 8, 2, D, Dv, x8=x8)
    c.check(*c.run(uniform=True))


@pytest.mark.parametrize("D,Dv", DIMS)
@pytest.mark.parametrize("x8", [False, True])
@pytest.mark.parametrize("page", [16, 64, 256])
def test_trees(D, Dv, x8, page):
    ns = [5, 1, 16, 0, 9]
    c = Case([100, 0, 333, 50, 64], ns, 4, 2, D, Dv, page=page, x8=x8, words=_tree(ns), pad=8)
    c.check(*c.run())


@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (5, 5), (16, 1), (12, 4), (64, 8), (48, 1)])
@pytest.mark.parametrize("n", [1, 3])
def test_groups(Hq, Hkv, n):
    c = Case([200, 70], [n, n], Hq, Hkv, 64, 64)
    c.check(*c.run(uniform=True))


@pytest.mark.parametrize("n", [2, 17, 33, 63, 64])
@pytest.mark.parametrize("chain", [True, False])
def test_many_drafted_tokens(n, chain):
    """Up to 64 a sequence, at every place of a tile; 64 x 8 rows are several row tiles."""
    ns = [n, n, n]
    c = Case([40, 0, 121], ns, 16, 2, 64, 64, page=32, words=None if chain else _tree(ns, n))
    c.check(*c.run(uniform=n % 2 == 0), heads=[0, 7, 9])


def test_empty_words_and_bits_behind_the_last_token():
    words = [0, 1 << 63 | 1, (1 << 64) - 1, 0]
    c = Case([0, 30], [2, 2], 2, 1, 64, 64, words=words)
    out, lse = c.run()
    c.check(out, lse)
    assert (out[0] == 0).all() and torch.isneginf(lse[0]).all()


@pytest.mark.parametrize("D,Dv", DIMS)
@pytest.mark.parametrize("x8", [False, True])
@pytest.mark.parametrize("group,n", [(2, 16), (2, 17), (2, 32), (2, 33), (2, 64), (5, 12), (5, 13), (5, 27)])
def test_rows_of_a_block(D, Dv, x8, group, n):
    """Rows around 32, 64 and 128: one block or two of 32, one of 128 or two; a second, shorter sequence leaves some idle."""
    ns = [n, 1, max(n - 9, 2)]
    c = Case([333, 5, 130], ns, 2 * group, 2, D, Dv, page=32, x8=x8, words=_tree(ns))
    c.check(*c.run())


@pytest.mark.parametrize("x8", [False, True])
@pytest.mark.parametrize("n", [1, 20])
def test_bad_pages_are_seen_by_nobody(x8, n):
    c = Case([100, 64, 130], [n] * 3, 4, 2, 64, 64, x8=x8)
    c.table[0, 2], c.table[0, 5], c.table[1, :], c.table[2, 0] = 10 ** 6, -7, -1, c.k.shape[0]
    c.pages = torch.tensor(c.table, device=DEV)
    out, lse = c.run()
    c.check(out, lse)
    assert (out[n:2 * n] == 0).all() and torch.isneginf(lse[n:2 * n]).all()


def test_contexts_behind_the_table_and_negative_ones():
    c = Case([40, -3], [8, 2], 2, 1, 64, 64)             # 48 places: whole pages, none of them unused
    c.dlens = torch.tensor([10 ** 9, -3], dtype=torch.int32, device=DEV)
    out, lse = c.run()
    c.lens = [16 * c.table.shape[1], -3]
    c.check(out, lse)


def test_rows_behind_max_q_and_behind_the_last_sequence():
    c = Case([40, 90], [5, 2], 2, 1, 64, 64)
    full, _ = c.run()
    out, lse = c.run(max_q=3)
    assert torch.equal(out[:3], full[:3]) and (out[3:5] == 5.0).all() and torch.equal(out[5:], full[5:])
    c.cu[2] = 6
    out, lse = c.run()
    assert torch.equal(out[:5], full[:5]) and (out[6:] == 5.0).all() and (lse[6:] == 5.0).all()


@pytest.mark.parametrize("B", [70, 200])
def test_many_sequences(B):
    """More than a wave's lanes, most of them short, a long one among them: runs that hold many and cut one."""
    lens = [(11 * b) % 90 for b in range(B)]
    lens[B // 2] = 5000
    ns = [b % 3 for b in range(B)]
    c = Case(lens, ns, 2, 1, 64, 64, words=_tree(ns))
    c.check(*c.run(), heads=[1], seqs=set(range(0, B, 7)) | {B // 2, B // 2 + 1, B - 1})


@pytest.mark.parametrize("x8", [False, True])
@pytest.mark.parametrize("Hkv", [1, 4])
def test_long_contexts_are_split_and_joined(x8, Hkv):
    c = Case([40000, 9, 7000], [1, 1, 1], 4 * Hkv, Hkv, 128, 128, page=64, x8=x8, sharp=4.0)
    c.check(*c.run(uniform=True), heads=[0, 4 * Hkv - 1])
    ns = [3, 40]
    c = Case([20000, 300], ns, 8, 1, 64, 64, page=128, x8=x8, words=_tree(ns))
    c.check(*c.run(), heads=[0, 7])


@pytest.mark.parametrize("D,Dv", DIMS)
def test_what_is_not_seen_has_no_influence(D, Dv):
    ns = [6, 4]
    words = [1, 3, 5, 8, 24, 33, 1, 2, 4, 8]
    c = Case([70, 200], ns, 4, 2, D, Dv, words=words)
    clean, lse = c.run()
    c.check(clean, lse)
    for bad in (float("nan"), float("inf")):
        p = 70 + 2                                       # drafted token 2 of the first sequence: seen by itself only
        page, row = c.table[0, p // 16], p % 16
        kc, vc = c.cache["kc"].clone(), c.cache["vc"].clone()
        vc[page, :, row] = bad
        kc[page, 1, row] = bad
        keep = dict(c.cache)
        c.cache.update(kc=kc, vc=vc)
        out, l2 = c.run()
        c.cache = keep
        torch.cuda.synchronize()
        assert not torch.isfinite(out[2].float()).any()
        rest = [i for i in range(10) if i != 2]
        assert torch.equal(out[rest], clean[rest]) and torch.equal(l2[rest], lse[rest])


def test_scale_byte_255_drops_its_group():
    c = Case([50], [1], 2, 1, 64, 64, x8=True)
    p = 13
    page = c.table[0, 0]
    c.cache["vs"][page, 0, p, 1] = 255
    c.cache["vc"][page, 0, p, 40] = 0x7f                 # NaN in a dropped group
    c.cache["ks"][page, 0, p, 0] = 255
    c.v[page, 0, p, 32:] = 0.0
    c.k[page, 0, p, :32] = 0.0
    c.check(*c.run())


def test_one_workspace_same_bits_streams_and_graphs():
    a = Case([3000, 10], [1, 1], 8, 2, 128, 128, page=64, seed=1)
    ns = [30, 11]
    b = Case([900, 2500], ns, 8, 2, 128, 128, x8=True, words=_tree(ns), seed=2)
    ws = k3.tree_attention_workspace(8, 2, 128, 64, device=DEV)
    wa, _ = a.run(uniform=True)
    wb, _ = b.run(max_q=64)
    a.check(wa, None, heads=[3])
    ws.fill_(0xff)                                       # what a workspace holds does not matter
    for _ in range(2):
        assert torch.equal(a.run(uniform=True, ws=ws)[0], wa)
        assert torch.equal(b.run(ws=ws, max_q=64)[0], wb)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    oa, ob = torch.zeros_like(wa), torch.zeros_like(wb)
    a.run(uniform=True, ws=ws, out=oa, lse=False, stream=s)
    s.synchronize()
    assert torch.equal(oa, wa)
    # words are made on the host by run(): the graph's tensors are held here
    tree = torch.tensor(b.words, dtype=torch.int64, device=DEV)
    graphs = [torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()]
    with torch.cuda.graph(graphs[0]):
        k3.tree_attention(a.q, pages=a.pages, lens=a.dlens, out=oa, workspace=ws, **a.cache)
    with torch.cuda.graph(graphs[1]):
        k3.tree_attention(b.q, pages=b.pages, lens=b.dlens, out=ob, cu_q=b.cu, max_q=64, tree=tree, workspace=ws, **b.cache)
    for step in range(3):
        a.dlens[0] -= 700                                # another context in the same graph
        want, _ = a.run(uniform=True)
        oa.zero_(), ob.zero_()
        graphs[0].replay()
        graphs[1].replay()
        torch.cuda.synchronize()
        assert torch.equal(oa, want) and torch.equal(ob, wb)


def test_two_calls_at_once_with_a_workspace_each():
    cases = [Case([4000 + 500 * i], [1], 8, 2, 64, 64, seed=i) for i in range(3)]
    want = [c.run()[0] for c in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    outs = [torch.zeros_like(w) for w in want]
    for _ in range(5):
        for c, s, o in zip(cases, streams, outs):
            c.run(out=o, lse=False, stream=s)            # workspace None: one of the call's own
    torch.cuda.synchronize()
    for o, w in zip(outs, want):
        assert torch.equal(o, w)


def test_a_cache_beyond_32_bits():
    pages, Hkv, page, D = 140000, 2, 64, 128
    if torch.cuda.mem_get_info()[0] < 2 * pages * Hkv * page * D * 2 + 2 ** 30:
        pytest.skip("not enough device memory")
    kc, vc = (torch.zeros((pages, Hkv, page, D), dtype=BF, device=DEV) for _ in range(2))
    assert kc.numel() * 2 > 2 ** 32
    c = Case([150], [1], 4, 2, D, D, page=page)
    for n, x in (("kc", kc), ("vc", vc)):
        x[pages - c.cache[n].shape[0]:] = c.cache[n]
        c.cache[n] = x
    c.pages += (pages - c.k.shape[0]) * (c.pages >= 0)
    out, lse = c.run()
    c.check(out, lse)


def test_two_streams_without_a_workspace():
    """Calls on the current stream and on another in turn, each with a workspace of its own making: the first one's is
    freed while its kernels run, and must not be the second one's."""
    a = Case([9000] * 12, [1] * 12, 16, 8, 64, 64, page=64, seed=1)
    b = Case([4000], [1], 16, 8, 64, 64, page=64, seed=2)
    wa, wb = a.run(uniform=True, lse=False)[0], b.run(uniform=True, lse=False)[0]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    outs = [(torch.zeros_like(wa), torch.zeros_like(wb)) for _ in range(6)]
    torch.cuda.synchronize()
    for oa, ob in outs:
        a.run(uniform=True, lse=False, out=oa)
        b.run(uniform=True, lse=False, out=ob, stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(oa, wa) and torch.equal(ob, wb) for oa, ob in outs)


@pytest.mark.parametrize("D,Dv", DIMS)
@pytest.mark.parametrize("x8", [False, True])
@pytest.mark.parametrize("n", [1, 8, 16, 64])
def test_a_workspace_of_the_stated_size_is_enough(D, Dv, x8, n):
    """Cut ends in every run: nothing behind the workspace is written."""
    c = Case([40000, 9000, 3], [n, n, 1], 8, 2, D, Dv, page=64, x8=x8)
    want = c.run(lse=False)[0]
    size = k3._tree_bytes(8, 2, Dv, n)
    buf = torch.full((size + 2 ** 20,), 0xab, dtype=torch.uint8, device=DEV)
    assert buf.data_ptr() % 256 == 0
    out = c.run(lse=False, ws=buf[:size])[0]
    assert torch.equal(out, want) and (buf[size:] == 0xab).all()

"""The paged cache: ttcd_paged_kv_append and ttcd_paged_window_attn against the
float64 oracle, with everything that a call must not read or write planted with
NaN: rows of pages behind a sequence, pages between the sinks and the window,
pages of nobody."""
import numpy as np
import pytest
import torch

from oracle import sink_oracle as so
from tests.helpers import np64
from tests.test_gpu_sink_attention import _within
from ttcd_workloads import make_attention_inputs

pytestmark = pytest.mark.gpu

NAN = float("nan")


@pytest.fixture(scope="module")
def ttcd():
    import dual_window_attention_b200 as m
    m.load_library()
    return m


class Batch:
    """Sequences with `lens` keys and `new` new tokens each; K and V of the whole
    sequences (dense, for the oracle) and the cache that holds what is seen."""

    def __init__(self, lens, new, Hq, Hkv, hd, page, window, n_sink, pad=0, seed=0, junk=None):
        g = torch.Generator().manual_seed(seed)
        self.lens, self.new, self.page, self.window, self.n_sink = lens, new, page, window, n_sink
        self.Hq, self.Hkv, self.hd, self.total = Hq, Hkv, hd, sum(new) + pad
        self.q = torch.randn(self.total, Hq, hd, generator=g).bfloat16()
        self.k = [torch.randn(L, Hkv, hd, generator=g).bfloat16() for L in lens]
        self.v = [torch.randn(L, Hkv, hd, generator=g).bfloat16() for L in lens]
        seen, self.kept = [], []
        for L, n in zip(lens, new):
            see = so.mask(np.arange(L - n, L), np.arange(L), window, n_sink).any(0) if n else np.zeros(L, bool)
            seen.append(see)
            self.kept.append(sorted({j // page for j in np.flatnonzero(see)}))
        n_pages = sum(map(len, self.kept)) + 4
        order = torch.randperm(n_pages, generator=g).tolist()
        table = torch.full((len(lens), max(-(-L // page) for L in lens) + 1), -1, dtype=torch.int32)
        if junk is not None:  # released entries may hold anything
            table.fill_(junk)
        k_pages = torch.full((n_pages, Hkv, page, hd), NAN).bfloat16()
        v_pages = k_pages.clone()
        for s, pages in enumerate(self.kept):
            for p in pages:
                table[s, p] = order.pop()
                a, b = p * page, min((p + 1) * page, lens[s])
                rows = torch.from_numpy(seen[s][a:b])
                for pool, x in ((k_pages, self.k[s]), (v_pages, self.v[s])):
                    at = pool[table[s, p], :, :b - a]
                    at[:, rows] = x[a:b][rows].transpose(0, 1)
        self.table, self.k_pages, self.v_pages = table.cuda(), k_pages.cuda(), v_pages.cuda()
        self.q_start = torch.tensor(np.concatenate([[0], np.cumsum(new)]), dtype=torch.int32).cuda()
        self.kv_len = torch.tensor(lens, dtype=torch.int32).cuda()

    def attend(self, ttcd, max_q=None, **kw):
        return ttcd.paged_window_attn(self.q.cuda(), self.k_pages, self.v_pages, self.table,
                                      self.q_start, self.kv_len, self.window, self.n_sink,
                                      max_q=max(1, *self.new) if max_q is None else max_q, **kw)

    def check(self, o, lse):
        scale, G, row = self.hd ** -0.5, self.Hq // self.Hkv, 0
        for s, (L, n) in enumerate(zip(self.lens, self.new)):
            for h in range(self.Hq if n else 0):
                ro, rl, _, bo = so.attend(np64(self.q[row:row + n, h]), np64(self.k[s][:, h // G]),
                                          np64(self.v[s][:, h // G]), np.arange(L - n, L),
                                          np.arange(L), self.window, self.n_sink, scale)
                _within(o[row:row + n, h], ro, bo, ("o", s, h))
                _within(lse[h, row:row + n], rl, so.W + 2.0 ** -22 * np.abs(rl), ("lse", s, h))
            row += n


CASES = [
    # lens, new, Hq, Hkv, hd, page, window, n_sink
    ([1], [1], 2, 1, 64, 16, 4, 0),                               # the first token
    ([1, 2, 17, 16, 300], [1, 1, 1, 1, 1], 4, 2, 64, 16, 40, 4),  # decode, pages that just end
    ([1000, 3, 777], [1, 1, 1], 16, 8, 128, 64, 200, 4),          # window and sinks apart
    ([1500, 1499], [1, 1], 8, 1, 128, 128, 1, 1),                 # itself and the first token
    ([2000], [1], 16, 1, 128, 32, 1500, 100),                     # groups of 16, many sinks
    ([900, 40], [1, 1], 32, 1, 64, 16, 333, 0),                   # groups of 32
    ([500, 130, 20], [4, 3, 2], 8, 2, 64, 16, 100, 3),            # a few tokens each
    ([300], [300], 4, 2, 64, 16, 64, 4),                          # a whole prompt
    ([700, 129], [200, 129], 6, 2, 128, 16, 150, 5),              # chunks, groups of 3
    ([1300, 64], [131, 64], 15, 5, 64, 32, 500, 128),             # a tile of sinks
    ([800, 5, 600, 900], [1, 5, 257, 1], 16, 8, 128, 64, 300, 4), # a batch of both kinds
    ([256, 200, 300], [0, 100, 0], 4, 4, 128, 128, 77, 2),        # sequences without new tokens
    ([400, 100], [30, 100], 5, 1, 32, 16, 90, 6),                 # head_dim 32
    ([3000], [2], 3, 1, 32, 64, 2500, 9),                         # head_dim 32, few rows
    ([10, 90], [3, 80], 128, 1, 64, 16, 50, 1),                   # groups of 128
]


@pytest.mark.parametrize("junk", [None, 1 << 30])
@pytest.mark.parametrize("lens,new,Hq,Hkv,hd,page,window,n_sink", CASES)
def test_attention(ttcd, lens, new, Hq, Hkv, hd, page, window, n_sink, junk):
    b = Batch(lens, new, Hq, Hkv, hd, page, window, n_sink, seed=len(lens) + hd, junk=junk)
    o, lse = b.attend(ttcd, lse=True)
    torch.cuda.synchronize()
    assert ttcd.get_device_error()[0] == ttcd.OK
    b.check(o, lse)
    # max_q only chooses the kernel
    for max_q in (1, 1000):
        b.check(*b.attend(ttcd, max_q=max_q, lse=True))
    assert ttcd.get_device_error()[0] == ttcd.OK


def test_many_sequences(ttcd):
    """More sequences than a warp looks through at once, some without new tokens."""
    r = np.random.default_rng(0)
    lens = r.integers(1, 200, 150).tolist()
    new = [int(min(L, x)) for L, x in zip(lens, r.choice([0, 1, 1, 1, 2, 30], 150))]
    b = Batch(lens, new, 4, 2, 64, 16, 50, 4, seed=9)
    b.check(*b.attend(ttcd, lse=True))
    b.check(*b.attend(ttcd, lse=True, max_q=1))
    assert ttcd.get_device_error()[0] == ttcd.OK


@pytest.mark.parametrize("max_q", [1, 60])
def test_padding_rows_are_left_as_they_were(ttcd, max_q):
    b = Batch([90, 200], [60, 1], 4, 2, 64, 16, 50, 4, pad=37)
    b.q[61:] = NAN
    o = torch.full((98, 4, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((4, 98), 7.0, device="cuda")
    b.attend(ttcd, o=o, lse=lse, max_q=max_q)
    b.check(o, lse)
    assert (o[61:] == 7).all() and (lse[:, 61:] == 7).all()
    assert ttcd.get_device_error()[0] == ttcd.OK


@pytest.mark.parametrize("max_q", [1, 60])
def test_pages_and_lengths_that_cannot_be(ttcd, max_q):
    """They are skipped and reported; the other sequences are as without them."""
    b = Batch([90, 200, 120], [60, 1, 3], 4, 2, 64, 16, 50, 4)
    o, lse = b.attend(ttcd, lse=True, max_q=max_q)
    b.check(o, lse)
    for bad in (-1, b.k_pages.shape[0], 2 ** 31 - 1, -2 ** 31):
        keep = b.table[1].clone()
        b.table[1, 200 // 16 - 1] = bad  # in the window of sequence 1
        o2, lse2 = b.attend(ttcd, lse=True, max_q=max_q)
        assert ttcd.get_device_error()[0] == ttcd.ERR_INVALID_ARG
        assert ttcd.get_device_error()[0] == ttcd.OK  # read and cleared
        b.table[1] = keep
        at = torch.tensor([i for i in range(64) if i != 60])
        assert torch.equal(o2[at], o[at]) and torch.equal(lse2[:, at], lse[:, at])
        assert torch.isfinite(o2[60]).all()  # the page counts as zeros
    for bad in (0, -5, b.table.shape[1] * 16 + 1, 2 ** 31 - 1, -2 ** 31):
        b.kv_len[1] = bad
        o2 = torch.full_like(o, 7.0)
        b.attend(ttcd, o=o2, max_q=max_q)
        assert ttcd.get_device_error()[0] == ttcd.ERR_INVALID_ARG
        assert torch.equal(o2[at], o[at]) and (o2[60] == 7).all()
    b.kv_len[1] = 200
    for bad in ([0, 60, 59, 64], [0, 60, 61, 65], [0, -60, 61, 64], [5, 3, 2, 1],
                [2 ** 31 - 1, -2 ** 31, 2 ** 31 - 1, 0]):
        b.q_start.copy_(torch.tensor(bad, dtype=torch.int32))
        b.attend(ttcd, max_q=max_q)
        assert ttcd.get_device_error()[0] == ttcd.ERR_INVALID_ARG, bad
    b.q_start.copy_(torch.tensor([0, 60, 61, 64], dtype=torch.int32))
    b.check(*b.attend(ttcd, lse=True, max_q=max_q))
    assert ttcd.get_device_error()[0] == ttcd.OK


@pytest.mark.parametrize("new", [[1, 1, 1], [1, 40, 3]])
def test_capture_replays_with_other_lengths(ttcd, new):
    """One captured call serves other lengths and pages of the same batch."""
    args = dict(Hq=4, Hkv=2, hd=64, page=16, window=50, n_sink=4)
    b = Batch([90, 200, 120], new, **args)
    q, total = b.q.cuda(), b.total
    kp = torch.full((64, 2, 16, 64), NAN, dtype=torch.bfloat16, device="cuda")
    vp = kp.clone()
    table = torch.full((3, 16), -1, dtype=torch.int32, device="cuda")
    q_start, kv_len = torch.zeros(4, dtype=torch.int32, device="cuda"), torch.zeros(3, dtype=torch.int32, device="cuda")

    def load(x):
        q.copy_(x.q)
        kp[:len(x.k_pages)].copy_(x.k_pages)
        vp[:len(x.v_pages)].copy_(x.v_pages)
        table.fill_(-1)
        table[:, :x.table.shape[1]].copy_(x.table)
        q_start.copy_(x.q_start)
        kv_len.copy_(x.kv_len)

    load(b)
    o, lse = torch.empty_like(q), torch.empty(4, total, device="cuda")
    call = lambda: ttcd.paged_window_attn(q, kp, vp, table, q_start, kv_len, 50, 4,  # noqa: E731
                                          max_q=max(new), o=o, lse=lse)
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for lens, nw, seed in (([91, 201, 121], new, 3), ([46, 44, 240], new[::-1], 4)):
        x = Batch(lens, nw, seed=seed, **args)
        load(x)
        graph.replay()
        torch.cuda.synchronize()
        x.check(o, lse)
    assert ttcd.get_device_error()[0] == ttcd.OK


def test_two_calls_at_once(ttcd):
    b, c = Batch([900, 40], [1, 1], 8, 2, 128, 16, 333, 4), Batch([300, 700], [200, 90], 8, 2, 128, 64, 100, 4)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    got = [x.attend(ttcd, lse=True, stream=s) for x, s in ((b, s1), (c, s2), (b, s2), (c, s1))]
    torch.cuda.synchronize()
    for x, y in zip((b, c, b, c), got):
        x.check(*y)


def test_a_page_past_2_31_elements(ttcd):
    """Offsets into the pool pass 32 bits."""
    Hkv, page, hd = 8, 128, 128
    n_pages = (2 ** 31 + 2 ** 24) // (Hkv * page * hd)
    kp = torch.empty(n_pages, Hkv, page, hd, dtype=torch.bfloat16, device="cuda")
    vp = torch.empty_like(kp)
    g = torch.Generator().manual_seed(0)
    k, v = (torch.randn(page, Hkv, hd, generator=g).bfloat16() for _ in range(2))
    kp[-1], vp[-1] = k.transpose(0, 1), v.transpose(0, 1)
    table = torch.tensor([[n_pages - 1]], dtype=torch.int32, device="cuda")
    for n in (1, 50):
        q = torch.randn(n, 8, hd, generator=g).bfloat16()
        one = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
        o, _ = ttcd.paged_window_attn(q.cuda(), kp, vp, table, one(0, n), one(128), 1000, 0, max_q=n)
        for h in range(8):
            ro, _, _, bo = so.attend(np64(q[:, h]), np64(k[:, h]), np64(v[:, h]),
                                     np.arange(128 - n, 128), np.arange(128), 1000, 0, hd ** -0.5)
            _within(o[:, h], ro, bo, "o")
    x = torch.randn(1, 24 * hd, generator=g).bfloat16().cuda()
    ttcd.paged_kv_append(x, kp, vp, table, one(0, 1), one(128), 8, rope_theta=0.0)
    assert torch.equal(kp[-1, :, 127], x.view(24, hd)[8:16]) and torch.equal(vp[-1, :, 127], x.view(24, hd)[16:])
    assert torch.equal(kp[-1, :, :127].cpu(), k.transpose(0, 1)[:, :127])
    assert ttcd.get_device_error()[0] == ttcd.OK


@pytest.mark.parametrize("lens,new,Hq,Hkv,hd,page,theta", [
    ([1], [1], 2, 1, 64, 16, 1e4),
    ([5, 1000, 17, 40], [5, 1, 1, 30], 4, 2, 64, 16, 1e4),
    ([700, 0, 129], [700, 0, 129], 16, 8, 128, 64, 1e6),
    ([60000, 9], [2, 9], 6, 3, 32, 128, 1e4),     # far positions, head_dim 32
    ([1 << 22], [3], 2, 2, 128, 128, 1e4),        # positions of millions
    ([50, 60], [20, 1], 4, 1, 128, 32, 0.0),      # no rotation
])
def test_append(ttcd, lens, new, Hq, Hkv, hd, page, theta):
    g = torch.Generator().manual_seed(1)
    total, pad = sum(new), 3
    qkv = torch.randn(total + pad, (Hq + 2 * Hkv) * hd, generator=g).bfloat16()
    held = [list(range((L - n) // page, -(-L // page))) for L, n in zip(lens, new)]
    n_pages = sum(map(len, held)) + 2
    order = torch.randperm(n_pages, generator=g).tolist()
    table = torch.full((len(lens), max(-(-L // page) for L in lens)), -7, dtype=torch.int32)
    for s, h in enumerate(held):
        for p in h:
            table[s, p] = order.pop()
    kp, vp = (torch.randn(n_pages, Hkv, page, hd, generator=g).bfloat16() for _ in range(2))
    q = torch.full((total + pad, Hq, hd), 7.0, dtype=torch.bfloat16, device="cuda")
    kc, vc = kp.cuda(), vp.cuda()
    q_start = torch.tensor(np.concatenate([[0], np.cumsum(new)]), dtype=torch.int32).cuda()
    out = ttcd.paged_kv_append(qkv.cuda(), kc, vc, table.cuda(), q_start,
                               torch.tensor(lens, dtype=torch.int32).cuda(), Hq, rope_theta=theta, q=q)
    assert out is q and ttcd.get_device_error()[0] == ttcd.OK
    assert (q[total:] == 7).all()
    x = np64(qkv).reshape(total + pad, Hq + 2 * Hkv, hd)
    pos = np.concatenate([np.arange(L - n, L) for L, n in zip(lens, new)])
    rot = x[:total, :Hq + Hkv]
    rot = so.rotate(rot, pos, theta) if theta else rot
    # half a step of bf16, and 2^-20 of the pair: cos and sin in 32 bits (an angle
    # off by 2 pi 2^-25 at most), two products and a sum
    half = hd // 2
    big = np.maximum(np.abs(x[:total, :Hq + Hkv, :half]), np.abs(x[:total, :Hq + Hkv, half:]))
    tol = so.U * np.abs(rot) + 2.0 ** -20 * np.concatenate([big, big], -1)
    _within(q[:total], rot[:, :Hq], tol[:, :Hq], "q")
    row = 0
    for s, (L, n) in enumerate(zip(lens, new)):
        for p in range(L - n, L):
            at = table[s, p // page]
            _within(kc[at, :, p % page], rot[row, Hq:], tol[row, Hq:], "k")
            assert torch.equal(vc[at, :, p % page].cpu(), qkv[row].view(-1, hd)[Hq + Hkv:])
            kp[at, :, p % page], vp[at, :, p % page] = 0, 0
            kc[at, :, p % page], vc[at, :, p % page] = 0, 0
            row += 1
    assert torch.equal(kc.cpu(), kp) and torch.equal(vc.cpu(), vp)  # nothing else was written


def test_append_skips_and_reports_what_cannot_be(ttcd):
    g = torch.Generator().manual_seed(2)
    qkv = torch.randn(5, 4 * 64, generator=g).bfloat16().cuda()
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731

    def call(table, q_start, kv_len):
        kp = torch.zeros(4, 1, 16, 64, dtype=torch.bfloat16, device="cuda")
        vp, q = torch.zeros_like(kp), torch.full((5, 2, 64), 7.0, dtype=torch.bfloat16, device="cuda")
        ttcd.paged_kv_append(qkv, kp, vp, i32(*table), i32(*q_start), i32(*kv_len), 2, q=q)
        return kp, vp, q, ttcd.get_device_error()[0]

    good = ([[0, 1], [2, 3]], [0, 2, 5], [18, 20])
    kp, vp, q, st = call(*good)
    assert st == ttcd.OK and (q != 7).any(-1).all()
    for page in (-1, 4, 2 ** 31 - 1, -2 ** 31):
        k2, v2, q2, st = call([[0, page], [2, 3]], *good[1:])
        assert st == ttcd.ERR_INVALID_ARG and torch.equal(q2, q)
        assert (k2[1] == 0).all() and torch.equal(k2[3], kp[3]) and torch.equal(v2[3], vp[3])
    for L in (1, 33, -1, 2 ** 31 - 1):
        k2, v2, q2, st = call(good[0], good[1], [L, 20])
        assert st == ttcd.ERR_INVALID_ARG and (q2[:2] == 7).all() and torch.equal(q2[2:], q[2:])
        assert (k2[:2] == 0).all() and torch.equal(k2[3], kp[3])
    for qs in ([0, 6, 5], [0, 2, 6], [-1, 2, 5], [2 ** 31 - 1, -2 ** 31, 5]):
        assert call(good[0], qs, good[2])[3] == ttcd.ERR_INVALID_ARG


@pytest.mark.parametrize("Hq,Hkv,hd,page,window,n_sink", [(4, 2, 64, 16, 70, 4), (16, 8, 128, 64, 200, 9)])
def test_a_prompt_in_chunks_then_tokens_is_the_dense_attention(ttcd, Hq, Hkv, hd, page, window, n_sink):
    """Append and attend, chunk by chunk and then token by token, for two sequences
    at different points, with pages given back once no later token sees them: the
    rows are those of ttcd_sink_window_attn over the whole sequences."""
    T, B = 500, 2
    g = torch.Generator().manual_seed(3)
    qkv = torch.randn(B, T, (Hq + 2 * Hkv) * hd, generator=g).bfloat16().cuda()
    n_pages = 2 * (-(-(window + 140) // page) + -(-n_sink // page)) + 2
    kp = torch.full((n_pages, Hkv, page, hd), NAN, dtype=torch.bfloat16, device="cuda")
    vp = kp.clone()
    free, held = list(range(n_pages)), [{}, {}]
    done = [0, 0]
    outs = [[], []]
    steps = [(130, 0), (7, 99), (0, 130), (1, 1), (100, 1), (1, 60)] + [(1, 1)] * 12
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    rot_q, rot_k = [[], []], [[], []]
    for step in steps:
        for s, n in enumerate(step):
            first = max(0, done[s] - window + 1)
            for p in [p for p in held[s] if (p + 1) * page <= first and p * page >= n_sink]:
                at = held[s].pop(p)
                kp[at], vp[at] = NAN, NAN
                free.append(at)
            for p in range(done[s] // page, -(-(done[s] + n) // page)):
                if p not in held[s]:
                    held[s][p] = free.pop()
        table = [[held[s].get(p, -1) for p in range(-(-T // page))] for s in range(B)]
        args = (i32(table), i32([0, step[0], step[0] + step[1]]), i32([done[s] + step[s] for s in range(B)]))
        x = torch.cat([qkv[s, done[s]:done[s] + step[s]] for s in range(B)])
        q = ttcd.paged_kv_append(x, kp, vp, *args, Hq)
        o, _ = ttcd.paged_window_attn(q, kp, vp, *args, window, n_sink, max_q=max(step))
        row = 0
        for s, n in enumerate(step):
            outs[s].append(o[row:row + n])
            rot_q[s].append(q[row:row + n])
            for p in range(done[s], done[s] + n):
                rot_k[s].append(kp[held[s][p // page], :, p % page].clone())
            done[s] += n
            row += n
    assert ttcd.get_device_error()[0] == ttcd.OK
    for s in range(B):
        n = done[s]
        q, k = torch.cat(rot_q[s])[None], torch.stack(rot_k[s])[None]
        v = qkv[s, :n].view(1, n, -1, hd)[:, :, Hq + Hkv:].contiguous()
        dense, _ = ttcd.sink_window_attn(q, k, v, window, n_sink)
        got = torch.cat(outs[s])
        ro, _, bo = so.sink_window_attention(np64(q), np64(k), np64(v), window, n_sink, hd ** -0.5)
        _within(got[None], ro, bo, "paged")
        _within(dense, ro, bo, "dense")

"""The cache ops (fr_attention_tree, fr_attention_weights, fr_cache_commit, fr_cache_evict) against their
definitions in 64 bits.

Tolerances, per element.  Products of bf16 values are exact in float32; a dot product of dh terms that is
summed in float32 is off by at most dh * 2^-24 * sum|q_d k_d| (delta after the scale).  Then
  lse  delta + (8 + |lse|) * 2^-21: the exponentials' approximation, the running sums, the conversions
       between base 2 and e, each a few float32 roundings of values up to |lse|;
  o    2^-8 |o| for the rounding of the output and 2^-8 sum p|v| for that of each p to bf16 (half a bf16
       step each), and sum p|v| * 2 * (lse's tolerance) for the relative error of each p;
  acc  w * (lse's tolerance + rows * 2^-24) for the weights' sum, 2^-23 of the result for the last add.
Where the ops run on each other's results, 2^-13 of the weight covers this: at dh = 64 sum|q_d k_d| / 8 is below
24, so that delta < 64 * 24 * 2^-24 < 2^-13.4, and the other terms are below 2^-16 together.
Slots past the drafted tokens hold NaN in every test, and outputs that must stay as they were a marker.
"""
import numpy as np
import pytest

from tests import _cache as R

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

import flow_matching_action_loop_b200 as fr  # noqa: E402

MARK = 7.0


def stream():
    return torch.cuda.current_stream().cuda_stream


def ptr(t):
    return 0 if t is None else t.data_ptr()


def seen_of(kind, B, N, rng):
    """[B][N][N] truth values, or None for the default sequence."""
    if kind == "chain":
        return None
    if kind == "none":
        return np.zeros((B, N, N), bool)
    if kind == "random":   # any bits, rows that see nothing among them
        s = rng.random((B, N, N)) < 0.4
        s[:, ::3] = False
        return s
    out = []
    for _ in range(B):
        parents = [int(rng.integers(-1, i)) if i else -1 for i in range(N)]
        out.append(R.sees(fr.fr_tree_mask(parents), N))
    return np.stack(out)


class Case:
    def __init__(self, B, Hq, Hkv, dh, N, S_max, lens, kind, seed=0, scale=1.5):
        rng = np.random.default_rng(seed + 1000 * N + S_max)
        self.B, self.Hq, self.Hkv, self.dh, self.N, self.S, self.lens = B, Hq, Hkv, dh, N, S_max, lens
        g = torch.Generator().manual_seed(seed + N + S_max)
        self.q = (torch.randn(B, Hq, N, dh, generator=g) * scale).bfloat16()
        self.k = torch.randn(B, Hkv, S_max, dh, generator=g).bfloat16()
        self.v = torch.randn(B, Hkv, S_max, dh, generator=g).bfloat16()
        for b, n in enumerate(lens):
            self.k[b, :, max(n, 0) + N if n >= 0 else 0:] = float("nan")
            self.v[b, :, max(n, 0) + N if n >= 0 else 0:] = float("nan")
        seen = seen_of(kind, B, N, rng)
        self.words = None if seen is None else np.stack([R.words_of(s) for s in seen])
        self.rng = rng

    def device(self):
        self.dq, self.dk, self.dv = self.q.cuda(), self.k.cuda(), self.v.cuda()
        self.dlens = torch.tensor(self.lens, dtype=torch.int32, device="cuda")
        self.dwords = None if self.words is None else torch.from_numpy(self.words.view(np.int32)).cuda()
        self.o = torch.full((self.B, self.N, self.Hq * self.dh), MARK, dtype=torch.bfloat16, device="cuda")
        self.lse = torch.full((self.B, self.Hq, self.N), MARK, device="cuda")
        self.nscratch = fr.fr_attention_tree_scratch_bytes(self.B, self.Hq, self.Hkv, self.N, self.S, self.dh)
        # a fresh workspace holds anything
        self.scratch = torch.full((max(self.nscratch, 16),), 0xFF, dtype=torch.uint8, device="cuda")
        return self

    def run(self):
        fr.fr_attention_tree(ptr(self.dq), ptr(self.dk), ptr(self.dv), ptr(self.dlens), ptr(self.dwords), ptr(self.o),
                             ptr(self.lse), self.B, self.Hq, self.Hkv, self.N, self.S, self.dh, ptr(self.scratch),
                             self.nscratch, stream())

    def oracle(self):
        return R.attend(self.q.double().numpy(), self.k.double().numpy(), self.v.double().numpy(), self.lens, self.words)


def check(c, o, lse, oracle=None):
    want, pv, wlse, size = oracle or c.oracle()
    got = o.float().cpu().numpy().reshape(want.shape).astype(np.float64)
    glse = lse.cpu().numpy().astype(np.float64)
    for b, n in enumerate(c.lens):
        if n < 0:
            assert np.all(got[b] == MARK) and np.all(glse[b] == MARK)
            continue
        empty = np.isinf(wlse[b])
        assert np.array_equal(glse[b] == -np.inf, empty)
        fin = np.where(empty, 0.0, wlse[b])
        tl = c.dh * 2.0 ** -24 * size[b] + (8 + np.abs(fin)) * 2.0 ** -21
        d = np.abs(np.where(empty, 0.0, glse[b]) - fin)
        assert np.all(d <= tl), (b, d.max(), tl.min())
        tol = 2.0 ** -8 * (np.abs(want[b]) + pv[b]) + pv[b] * 2 * tl.T[:, :, None] + 1e-30
        d = np.abs(got[b] - want[b])
        assert np.all(d <= tol), (b, float(d.max()), np.unravel_index(np.argmax(d - tol), d.shape))


ATTEND = [
    # B, Hq, Hkv, dh, N, S_max, lens, mask
    (1, 1, 1, 64, 1, 1, [0], "chain"),                        # one token that sees itself alone
    (1, 8, 1, 256, 1, 866, [816], "chain"),                   # the backbone's heads over one prefix
    (2, 4, 2, 128, 1, 2, [0, 1], "none"),                     # nothing to see; one committed slot
    (3, 2, 1, 64, 5, 140, [127, -1, 0], "tree"),              # a padded sample between others
    (4, 16, 2, 128, 24, 160, [128, 129, 127, 136], "tree"),   # tiles that end at, before and after the drafts
    (2, 8, 1, 256, 33, 300, [200, 31], "random"),             # rows that see no drafted token
    (2, 8, 1, 256, 17, 17, [0, 0], "random"),                 # rows that see nothing at all
    (1, 3, 3, 64, 256, 700, [444], "tree"),                   # as many drafted tokens as there may be
    (1, 4, 1, 64, 256, 513, [257], "chain"),                  # eight row tiles, a sequence
    (2, 7, 1, 128, 19, 515, [496, 300], "tree"),              # a group of seven, 133 rows
    (5, 12, 4, 64, 3, 130, [1, 2, 60, 127, -5], "tree"),
    (9, 2, 2, 128, 2, 1000, [0, 998, 5, 640, 127, 128, 384, 900, 1], "chain"),   # ragged
    (1, 2, 1, 64, 2, 40000, [39998], "chain"),                # long
    (1, 8, 1, 256, 16, 5000, [4800], "tree"),                 # 128 rows, many tiles
    (40, 8, 8, 64, 1, 200, [150 + i % 40 for i in range(40)], "chain"),          # more units than SMs
    (33, 5, 5, 128, 4, 300, [(37 * i) % 297 for i in range(33)], "tree"),
    # several tiles per CTA, segments that begin and end inside units, several row tiles
    (3, 8, 1, 256, 63, 9000, [8900, 7001, 8555], "tree"),
    (30, 4, 2, 256, 3, 3000, [2990 - 31 * i for i in range(30)], "tree"),
    (12, 6, 2, 128, 130, 2300, [2100, -1, 2000, 300, 0, 2170, 1999, 5, 1500, 700, 2048, 129], "tree"),
    (2, 34, 1, 64, 64, 6000, [5900, 3333], "chain"),          # 17 row tiles: two batches
    # single tokens over a cache that streams from memory: tiles land late and out of order
    (24, 32, 8, 128, 1, 4200, [4190 - 97 * i for i in range(24)], "chain"),
    # short units whole, long ones cut, in one call
    (70, 8, 1, 128, 16, 2600, [[100, 2584, 0, 700, -1, 1900, 511, 33][i % 8] for i in range(70)], "tree"),
    (160, 2, 2, 64, 3, 900, [(211 * i) % 898 for i in range(160)], "random"),
    (90, 8, 1, 256, 24, 1100, [1076 - 5 * i for i in range(90)], "tree"),
]


@pytest.mark.parametrize("spec", ATTEND, ids=lambda s: "-".join(map(str, s[:6])) + "-" + s[7])
def test_tree_attention(spec):
    c = Case(*spec).device()
    c.run()
    first = (c.o.clone(), c.lse.clone())
    check(c, *first)
    c.run()   # the workspace as the first call left it: the same bits
    assert torch.equal(c.o, first[0]) and torch.equal(c.lse, first[1])
    assert fr.fr_ops_sync_status(stream()) == 0


@pytest.mark.parametrize("dh", [64, 128, 256])
def test_tree_attention_large_scores(dh):
    """Scores of both signs up to hundreds, growing along the cache: the running maximum moves in many tiles."""
    c = Case(1, 4, 1, dh, 9, 900, [800], "tree", seed=3, scale=6.0)
    c.k[0, 0, :809] *= torch.linspace(0.05, 4.0, 809)[:, None].to(torch.bfloat16)
    c.device().run()
    check(c, c.o, c.lse)


def test_tree_attention_hidden_values_do_not_leak():
    """A drafted token with NaN or infinite K and V reaches the rows that see it and no others."""
    c = Case(1, 8, 1, 128, 40, 400, [301], "chain")
    hidden = [3, 17, 39]
    seen = np.tril(np.ones((40, 40), bool))
    seen[:, hidden] = False
    seen[hidden, hidden] = True
    c.words = R.words_of(seen)[None]
    oracle = c.oracle()
    c.k[0, 0, 301 + 3], c.v[0, 0, 301 + 3] = float("nan"), float("nan")
    c.k[0, 0, 301 + 17], c.v[0, 0, 301 + 17] = float("inf"), float("-inf")
    c.v[0, 0, 301 + 39, 5] = float("inf")
    c.device().run()
    got = c.o.view(40, 8, 128).float()
    for i in hidden:
        assert torch.isnan(got[i]).all()
        c.o.view(40, 8, 128)[i] = torch.from_numpy(oracle[0][0, i]).cuda().bfloat16()
        c.lse[0, :, i] = torch.from_numpy(oracle[2][0, :, i]).cuda().float()
    check(c, c.o, c.lse, oracle)


@pytest.mark.parametrize("dh", [64, 128, 256])
def test_tree_attention_hidden_values_in_a_large_batch(dh):
    """The same in every third sample of a batch that is shared over the whole GPU."""
    B, N = 60, 20
    c = Case(B, 8, 4, dh, N, 700, [20 + 11 * b for b in range(B)], "chain")
    seen = np.tril(np.ones((N, N), bool))
    seen[:, 7] = False
    seen[7, 7] = True
    c.words = np.stack([R.words_of(seen)] * B)
    oracle = c.oracle()
    for b in range(0, B, 3):
        c.k[b, :, c.lens[b] + 7] = float("inf")
        c.v[b, 1:, c.lens[b] + 7, 5] = float("nan")
        c.v[b, 0, c.lens[b] + 7] = float("-inf")
    c.device().run()
    o = c.o.view(B, N, 8, dh)
    for b in range(0, B, 3):
        assert torch.isnan(o[b, 7]).all()
        o[b, 7] = torch.from_numpy(oracle[0][b, 7]).cuda().bfloat16()
        c.lse[b, :, 7] = torch.from_numpy(oracle[2][b, :, 7]).cuda().float()
    check(c, c.o, c.lse, oracle)


# a unit alone, split over a cluster, over CTAs of many units, of several row tiles
@pytest.mark.parametrize("spec", [(1, 4, 2, 64, 5, 100, [60]), (2, 8, 1, 256, 7, 3000, [2900, 2500]), (1, 2, 1, 128, 130, 5000, [4700]),
                                  (40, 4, 4, 128, 5, 900, [880 - 7 * b for b in range(40)])], ids=lambda s: "-".join(map(str, s[:6])))
def test_a_query_that_is_not_finite_spoils_its_own_row_alone(spec):
    c = Case(*spec, "tree").device()
    c.run()
    o, lse = c.o.clone().view(c.B, c.N, c.Hq, c.dh), c.lse.clone()
    at = [(0, 0, 0), (c.B - 1, c.Hq - 1, c.N - 1), (0, c.Hq // 2, c.N // 2)]
    for b, h, i in at:
        c.dq[b, h, i] = float("nan")
    c.run()
    o2 = c.o.view(o.shape)
    rest = torch.ones(c.B, c.Hq, c.N, dtype=torch.bool, device="cuda")
    for b, h, i in at:
        assert torch.isnan(o2[b, i, h]).all() and torch.isnan(c.lse[b, h, i])
        rest[b, h, i] = False
    assert torch.equal(o2.transpose(1, 2)[rest], o.transpose(1, 2)[rest]) and torch.equal(c.lse[rest], lse[rest])


@pytest.mark.parametrize("dh", [64, 128, 256])
def test_weights_of_rows_that_are_not_finite(dh):
    """Rows out of use may hold anything; a NaN row reaches the slots that it sees, no others."""
    B, Hq, Hkv, N, S, lens = 2, 80, 2, 9, 700, [600, 77]
    c = Case(B, Hq, Hkv, dh, N, S, lens, "tree").device()
    _, _, lse, _ = c.oracle()
    use = np.full((B, 1), 0x1ff & ~0x24, np.uint32)     # tokens 2 and 5 do not count
    d_use, d_lse = torch.from_numpy(use.view(np.int32)).cuda(), torch.from_numpy(lse).float().cuda()

    def weights():
        acc = torch.zeros(B, Hkv, S, device="cuda")
        fr.fr_attention_weights(ptr(c.dq), ptr(c.dk), ptr(d_lse), ptr(c.dlens), ptr(c.dwords), ptr(d_use), ptr(acc), B, Hq, Hkv, N, S,
                                dh, stream())
        return acc

    want = weights()
    for v in (float("nan"), float("inf")):
        c.dq[:, ::3, 2], c.dq[:, :, 5] = v, -v
        d_lse[:, ::3, 2], d_lse[:, ::2, 5] = float("nan"), v
        assert torch.equal(weights(), want)
    d_lse[1, 7, 3] = float("nan")                       # a row in use, of sample 1 and KV head 0
    got = weights()
    sees = np.concatenate([np.ones(lens[1], bool), R.sees(c.words[1], N)[3]])
    n = lens[1] + N
    assert torch.equal(torch.isnan(got[1, 0, :n]).cpu(), torch.from_numpy(sees))
    got[1, 0, :n][torch.from_numpy(sees).cuda()] = want[1, 0, :n][torch.from_numpy(sees).cuda()]
    assert torch.equal(got, want)


@pytest.mark.parametrize("dh", [64, 128, 256])
def test_tree_attention_large_scores_over_the_whole_gpu(dh):
    c = Case(20, 8, 8, dh, 3, 3000, [2900 - 7 * b for b in range(20)], "tree", seed=5, scale=5.0)
    for b in range(20):
        c.k[b, :, :c.lens[b]] *= torch.linspace(0.02, 3.0, c.lens[b])[None, :, None].to(torch.bfloat16)
    c.device().run()
    check(c, c.o, c.lse)


def test_tree_attention_in_a_cache_far_longer_than_its_sequences():
    c = Case(3, 8, 2, 128, 5, 60000, [100, 0, 700], "tree").device()
    c.run()
    check(c, c.o, c.lse)


def test_offsets_past_four_gigabytes():
    """K and V of 4.6 GB each: only the last sample, whose rows lie past 2^32 bytes, is in use."""
    B, Hq, Hkv, dh, N, S = 9, 16, 8, 64, 6, 520000
    if torch.cuda.mem_get_info()[0] < 24 << 30:
        pytest.skip("needs 24 GB")
    assert (B * Hkv - 1) * S * dh * 2 > 1 << 32
    c = Case(1, Hq, Hkv, dh, N, 400, [390], "tree")
    k, v = torch.empty(B, Hkv, S, dh, dtype=torch.bfloat16, device="cuda"), torch.empty(B, Hkv, S, dh, dtype=torch.bfloat16, device="cuda")
    k[-1, :, :400], v[-1, :, :400] = c.k[0].cuda(), c.v[0].cuda()
    lens = torch.full((B,), -1, dtype=torch.int32, device="cuda")
    lens[-1] = 390
    q = torch.zeros(B, Hq, N, dh, dtype=torch.bfloat16, device="cuda")
    q[-1] = c.q[0].cuda()
    words = torch.zeros(B, N, 1, dtype=torch.int32, device="cuda")
    words[-1] = torch.from_numpy(c.words[0].view(np.int32)).cuda()
    o, lse = torch.empty(B, N, Hq * dh, dtype=torch.bfloat16, device="cuda"), torch.empty(B, Hq, N, device="cuda")
    n = fr.fr_attention_tree_scratch_bytes(B, Hq, Hkv, N, S, dh)
    scratch = torch.empty(n, dtype=torch.uint8, device="cuda")
    fr.fr_attention_tree(ptr(q), ptr(k), ptr(v), ptr(lens), ptr(words), ptr(o), ptr(lse), B, Hq, Hkv, N, S, dh, ptr(scratch), n, stream())
    check(c, o[-1:], lse[-1:])
    acc, pos = torch.zeros(B, Hkv, S, device="cuda"), torch.zeros(B, Hkv, S, dtype=torch.int32, device="cuda")
    fr.fr_attention_weights(ptr(q), ptr(k), ptr(lse), ptr(lens), ptr(words), 0, ptr(acc), B, Hq, Hkv, N, S, dh, stream())
    want, _ = R.weigh(c.q.double().numpy(), c.k.double().numpy(), lse[-1:].double().cpu().numpy(), [390], c.words, None, np.zeros((1, Hkv, S)))
    assert np.all(np.abs(acc[-1].cpu().numpy() - want[0])[:, :396] <= 2.0 ** -13 * want[0][:, :396]) and float(acc[:-1].abs().max()) == 0.0
    path, npath = torch.zeros(B, N, dtype=torch.int32, device="cuda"), torch.full((B,), 3, dtype=torch.int32, device="cuda")
    path[-1] = torch.tensor([1, 2, 5, 0, 0, 0], dtype=torch.int32)
    lens2, lens3 = torch.empty_like(lens), torch.empty_like(lens)
    kk, vv = k[-1, :, :396].clone(), v[-1, :, :396].clone()
    fr.fr_cache_commit(ptr(k), ptr(v), 0, 0, ptr(lens), ptr(path), ptr(npath), ptr(lens2), B, Hkv, N, S, dh, fr.FR_DTYPE_BF16, stream())
    at = [391, 392, 395]
    assert lens2.tolist() == [-1] * (B - 1) + [393]
    assert torch.equal(k[-1, :, 390:393], kk[:, at]) and torch.equal(v[-1, :, 390:393], vv[:, at])
    kk, vv = k[-1, :, :393].clone(), v[-1, :, :393].clone()
    acc2, pos2, src = torch.zeros_like(acc), torch.zeros_like(pos), torch.zeros(B, Hkv, 100, dtype=torch.int32, device="cuda")
    fr.fr_cache_evict(ptr(k), ptr(v), ptr(acc), ptr(pos), ptr(lens2), ptr(acc2), ptr(pos2), ptr(lens3), ptr(src), B, Hkv, S, dh,
                      fr.FR_DTYPE_BF16, 100, 0, stream())
    assert lens3.tolist() == [-1] * (B - 1) + [100]
    for h in range(Hkv):
        at = R.evict_one(acc[-1, h, :393].cpu().numpy(), np.zeros(393, np.int32), 100, 0)
        assert src[-1, h].tolist() == at.tolist()
        t = torch.from_numpy(at).cuda()
        assert torch.equal(k[-1, h, :100], kk[h][t]) and torch.equal(v[-1, h, :100], vv[h][t])
    assert fr.fr_ops_sync_status(stream()) == 0


def test_the_four_ops_in_one_graph_over_the_whole_gpu():
    """Captured together at sizes that take the merge kernel; replayed on another state."""
    B, Hq, Hkv, dh, N, S, keep = 40, 16, 8, 128, 5, 900, 500
    a = Case(B, Hq, Hkv, dh, N, S, [890 - 20 * b for b in range(B)], "tree")
    b = Case(B, Hq, Hkv, dh, N, S, [95 + 20 * b for b in range(B)], "tree", seed=1)
    lens2, lens3 = torch.zeros(B, dtype=torch.int32).cuda(), torch.zeros(B, dtype=torch.int32).cuda()
    acc, acc2 = torch.zeros(B, Hkv, S).cuda(), torch.zeros(B, Hkv, S).cuda()
    pos = torch.arange(S, dtype=torch.int32).expand(B, Hkv, S).contiguous().cuda()
    pos2, src = torch.zeros_like(pos), torch.zeros(B, Hkv, keep, dtype=torch.int32).cuda()
    path = torch.tensor([0, 2, 3, 4, 4], dtype=torch.int32).expand(B, N).contiguous().cuda()
    npath = torch.tensor([i % 5 for i in range(B)], dtype=torch.int32).cuda()
    a.device(), b.device()

    def ops(c, s):
        fr.fr_attention_tree(ptr(c.dq), ptr(c.dk), ptr(c.dv), ptr(c.dlens), ptr(c.dwords), ptr(c.o), ptr(c.lse), B, Hq, Hkv, N, S,
                             dh, ptr(c.scratch), c.nscratch, s)
        fr.fr_attention_weights(ptr(c.dq), ptr(c.dk), ptr(c.lse), ptr(c.dlens), ptr(c.dwords), 0, ptr(acc), B, Hq, Hkv, N, S, dh, s)
        fr.fr_cache_commit(ptr(c.dk), ptr(c.dv), ptr(acc), ptr(pos), ptr(c.dlens), ptr(path), ptr(npath), ptr(lens2), B, Hkv, N, S,
                           dh, fr.FR_DTYPE_BF16, s)
        fr.fr_cache_evict(ptr(c.dk), ptr(c.dv), ptr(acc), ptr(pos), ptr(lens2), ptr(acc2), ptr(pos2), ptr(lens3), ptr(src), B, Hkv,
                          S, dh, fr.FR_DTYPE_BF16, keep, 8, s)

    def reset(c):
        c.dk.copy_(c.k), c.dv.copy_(c.v)
        acc.zero_(), acc2.zero_(), pos2.zero_(), src.zero_()
        pos.copy_(torch.arange(S, dtype=torch.int32).expand(B, Hkv, S))

    ops(b, stream())   # the answer of the plain calls on b's state
    want = [x.clone() for x in (b.o, b.lse, b.dk, b.dv, acc, pos, lens2, acc2, pos2, lens3, src)]
    check(b, b.o, b.lse)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    reset(a)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        ops(a, torch.cuda.current_stream().cuda_stream)
    graph.replay()
    check(a, a.o, a.lse)
    a.k, a.v = b.k, b.v
    a.dq.copy_(b.dq), a.dlens.copy_(b.dlens), a.dwords.copy_(b.dwords)
    for _ in range(2):
        reset(a)
        graph.replay()
        for x, y in zip((a.o, a.lse, a.dk, a.dv, acc, pos, lens2, acc2, pos2, lens3, src), want):
            assert torch.equal(torch.nan_to_num(x.float()), torch.nan_to_num(y.float()))
    assert fr.fr_ops_sync_status(stream()) == 0


def test_tree_attention_refuses_bad_lengths_on_the_device():
    c = Case(4, 4, 2, 64, 3, 100, [50, 97, 20, 4], "tree").device()
    c.dlens[0], c.dlens[2] = 98, 2 ** 31 - 1      # lens + N past the cache
    c.lens = [-1, 97, -1, 4]                      # the oracle's view: skipped samples
    c.run()
    check(c, c.o, c.lse)
    with pytest.raises(fr.FrError) as e:
        fr.fr_ops_sync_status(stream())
    assert e.value.code == fr.FR_ERR_DEVICE and "c001" in str(e.value)
    assert fr.fr_ops_sync_status(stream()) == 0


def test_tree_attention_without_lse_and_in_a_graph():
    """lse may be NULL; a captured call follows lens and mask as they change between replays."""
    c = Case(3, 8, 2, 128, 6, 700, [600, 30, -1], "tree").device()
    c.run()
    o = c.o.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        fr.fr_attention_tree(ptr(c.dq), ptr(c.dk), ptr(c.dv), ptr(c.dlens), ptr(c.dwords), ptr(c.o), 0, c.B, c.Hq, c.Hkv,
                             c.N, c.S, c.dh, ptr(c.scratch), c.nscratch, torch.cuda.current_stream().cuda_stream)
    c.o.fill_(MARK)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(c.o, o)
    c.lens = [100, -1, 17]
    c.dlens.copy_(torch.tensor(c.lens, dtype=torch.int32))
    c.words[:] = c.words[::-1].copy()
    c.dwords.copy_(torch.from_numpy(c.words.view(np.int32)))
    # the third sample's cache was padding; give it rows
    c.k[2, :, :23], c.v[2, :, :23] = c.k[0, :, :23], c.v[0, :, :23]
    c.dk.copy_(c.k), c.dv.copy_(c.v)
    c.o.fill_(MARK)
    graph.replay()
    want = c.o.clone()
    c.o.fill_(MARK), c.lse.fill_(MARK)
    c.run()
    assert torch.equal(c.o, want)
    check(c, c.o, c.lse)


def test_tree_attention_on_two_streams_with_their_own_workspaces():
    a, b = Case(2, 8, 1, 256, 9, 3000, [2500, 2900], "tree").device(), Case(2, 8, 1, 256, 9, 3000, [100, 1700], "tree", seed=9).device()
    torch.cuda.synchronize()
    s = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        for c, st in zip((a, b), s):
            with torch.cuda.stream(st):
                c.run()
    torch.cuda.synchronize()
    check(a, a.o, a.lse)
    check(b, b.o, b.lse)


WEIGH = [s for s in ATTEND if s[5] <= 9000 and s[0] not in (24, 70, 90, 160)]


@pytest.mark.parametrize("spec", WEIGH, ids=lambda s: "-".join(map(str, s[:6])) + "-" + s[7])
@pytest.mark.parametrize("some", [False, True])
def test_attention_weights(spec, some):
    c = Case(*spec).device()
    N = c.N
    use = None
    if some:
        use = np.zeros((c.B, -(-N // 32)), np.uint32)
        for b in range(c.B):
            for i in range(N):
                if c.rng.random() < 0.5:
                    use[b, i // 32] |= np.uint32(1 << (i % 32))
    _, _, lse, size = c.oracle()
    lse32 = torch.from_numpy(lse).float()
    acc = torch.rand(c.B, c.Hkv, c.S, generator=torch.Generator().manual_seed(5))
    d_acc, d_lse = acc.cuda(), lse32.cuda()
    d_use = None if use is None else torch.from_numpy(use.view(np.int32)).cuda()

    def call():
        fr.fr_attention_weights(ptr(c.dq), ptr(c.dk), ptr(d_lse), ptr(c.dlens), ptr(c.dwords), ptr(d_use), ptr(d_acc),
                                c.B, c.Hq, c.Hkv, N, c.S, c.dh, stream())
    call()
    want, w = R.weigh(c.q.double().numpy(), c.k.double().numpy(), lse32.double().numpy(), c.lens, c.words, use, acc.numpy())
    got = d_acc.cpu().numpy().astype(np.float64)
    rows = c.Hq // c.Hkv * N
    fin = np.where(np.isinf(lse), 0.0, np.abs(lse))
    tl = c.dh * 2.0 ** -24 * size.max() + (8 + fin.max()) * 2.0 ** -21
    for b, n in enumerate(c.lens):
        used = n + N if n >= 0 else 0
        assert np.array_equal(got[b, :, used:], acc[b, :, used:].double().numpy())
        d = np.abs(got[b, :, :used] - want[b, :, :used])
        assert np.all(d <= w[b, :, :used] * (tl + rows * 2.0 ** -24) + 2.0 ** -23 * want[b, :, :used] + 1e-37), d.max()
    once = d_acc.clone()
    d_acc.copy_(acc)
    call()
    assert torch.equal(d_acc, once)   # the same bits
    assert fr.fr_ops_sync_status(stream()) == 0


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("B,Hkv,dh,N,S,lens", [
    (1, 1, 256, 24, 866, [816]),
    (3, 2, 64, 1, 9, [0, 8, -1]),
    (4, 3, 128, 63, 200, [137, 0, 100, 50]),
    (2, 1, 512, 256, 600, [344, 1]),
    (2, 2, 8, 256, 300, [44, 0]),
    (1, 1, 24, 40, 41, [1]),
])
@pytest.mark.parametrize("optional", [True, False])
def test_commit(B, Hkv, dh, N, S, lens, dtype, optional):
    rng = np.random.default_rng(N + S)
    g = torch.Generator().manual_seed(N)
    k, v = torch.randn(B, Hkv, S, dh, generator=g).to(dtype), torch.randn(B, Hkv, S, dh, generator=g).to(dtype)
    acc, pos = torch.rand(B, Hkv, S, generator=g), torch.randint(0, 1 << 30, (B, Hkv, S), generator=g, dtype=torch.int32)
    for trial in range(4):
        npath = [[0, N, int(rng.integers(0, N + 1)), 1][(trial + b) % 4] for b in range(B)]
        path = np.full((B, N), -9, np.int32)   # entries past npath are not looked at
        for b in range(B):
            path[b, :npath[b]] = np.sort(rng.permutation(N)[:npath[b]])
        t = [x.clone() for x in (k, v, acc, pos)]
        out = lens[:]
        for b, n in enumerate(lens):
            if n < 0:
                continue
            at = n + path[b, :npath[b]].astype(np.int64)
            for x in t if optional else t[:2]:
                x[b, :, n:n + npath[b]] = x[b][:, torch.from_numpy(at)]
            out[b] = n + npath[b]
        dev = [x.cuda() for x in (k, v, acc, pos)]
        d_lens = torch.tensor(lens, dtype=torch.int32).cuda()
        d_path, d_np = torch.from_numpy(path).cuda(), torch.tensor(npath, dtype=torch.int32).cuda()
        d_out = torch.full((B,), 99, dtype=torch.int32, device="cuda")
        fr.fr_cache_commit(ptr(dev[0]), ptr(dev[1]), ptr(dev[2]) if optional else 0, ptr(dev[3]) if optional else 0,
                           ptr(d_lens), ptr(d_path), ptr(d_np), ptr(d_out), B, Hkv, N, S, dh,
                           fr.FR_DTYPE_F32 if dtype == torch.float32 else fr.FR_DTYPE_BF16, stream())
        for x, y in zip(dev, t):
            assert torch.equal(x.cpu(), y)
        assert d_out.tolist() == out
        assert fr.fr_ops_sync_status(stream()) == 0


def test_commit_refuses_bad_paths_on_the_device():
    B, Hkv, N, S, dh = 6, 2, 4, 50, 64
    k = torch.randn(B, Hkv, S, dh).cuda()
    v, k0 = k.clone() + 1, k.clone()
    lens = torch.tensor([10, 10, 10, 47, 10, 10], dtype=torch.int32).cuda()
    path = torch.tensor([[0, 2, 1, 3], [0, 1, 2, 4], [1, 1, 2, 3], [0, 1, 2, 3], [-1, 0, 1, 2], [1, 3, 0, 0]], dtype=torch.int32).cuda()
    npath = torch.tensor([3, 4, 2, 1, 1, 2], dtype=torch.int32).cuda()
    out = torch.zeros(B, dtype=torch.int32).cuda()
    fr.fr_cache_commit(ptr(k), ptr(v), 0, 0, ptr(lens), ptr(path), ptr(npath), ptr(out), B, Hkv, N, S, dh, fr.FR_DTYPE_F32, stream())
    assert out.tolist() == [10, 10, 10, 47, 10, 12]
    want = k0.clone()
    want[5, :, 10:12] = k0[5][:, [11, 13]]
    assert torch.equal(k, want) and torch.equal(v, want + 1)
    with pytest.raises(fr.FrError) as e:
        fr.fr_ops_sync_status(stream())
    assert e.value.code == fr.FR_ERR_DEVICE
    npath.copy_(torch.tensor([5, -1, 0, 0, 0, 0], dtype=torch.int32))
    lens[3] = -1
    fr.fr_cache_commit(ptr(k), ptr(v), 0, 0, ptr(lens), ptr(path), ptr(npath), ptr(out), B, Hkv, N, S, dh, fr.FR_DTYPE_F32, stream())
    assert out.tolist() == [10, 10, 10, -1, 10, 10] and torch.equal(k, want)
    with pytest.raises(fr.FrError) as e:
        fr.fr_ops_sync_status(stream())
    assert "c002" in str(e.value)


EVICT = [
    # B, Hkv, dh, S_max, lens, keep, recent, weights, dtype
    (1, 1, 256, 866, [866], 512, 50, "spread", "bf16"),
    (1, 1, 8, 1, [1], 1, 0, "spread", "bf16"),
    (3, 2, 64, 40, [0, 40, -1], 1, 1, "spread", "f32"),
    (4, 2, 64, 300, [299, 128, 129, 300], 128, 0, "ties", "bf16"),
    (4, 2, 64, 300, [299, 128, 129, 300], 128, 128, "spread", "f32"),     # every kept slot protected
    (2, 3, 128, 3000, [2999, 2050], 2049, 7, "few", "bf16"),
    (2, 1, 64, 9000, [9000, 6001], 600, 64, "ties", "bf16"),
    (1, 2, 64, 40001, [40001], 39999, 1000, "spread", "bf16"),
    (2, 1, 16, 70000, [70000, 69999], 10, 3, "odd", "f32"),
    (1, 1, 8, 524288, [524288], 262145, 100, "spread", "bf16"),           # as many slots as there may be
    (30, 4, 64, 500, [499 - 7 * i for i in range(30)], 333, 33, "few", "f32"),
    (2, 2, 512, 260, [250, 100], 99, 0, "equal", "f32"),
]


@pytest.mark.parametrize("B,Hkv,dh,S,lens,keep,recent,weights,dt", EVICT)
def test_evict(B, Hkv, dh, S, lens, keep, recent, weights, dt):
    rng = np.random.default_rng(S + keep)
    dtype = torch.float32 if dt == "f32" else torch.bfloat16
    g = torch.Generator(device="cuda").manual_seed(S)
    k = torch.randn(B, Hkv, S, dh, generator=g, device="cuda").to(dtype)
    v = torch.randn(B, Hkv, S, dh, generator=g, device="cuda").to(dtype)
    if weights == "spread":
        acc = np.exp(rng.standard_normal((B, Hkv, S)) * 3)
    elif weights == "ties":
        acc = rng.integers(0, 4, (B, Hkv, S)).astype(np.float64)
    elif weights == "few":
        acc = np.where(rng.random((B, Hkv, S)) < 0.02, 5.0, rng.random((B, Hkv, S)) * 2.0 ** -140)
    elif weights == "equal":
        acc = np.zeros((B, Hkv, S))
    else:   # signs, zeros of both signs, infinities, NaN
        acc = rng.choice([0.0, -0.0, -1.5, 2.0, np.inf, -np.inf, np.nan, 1e-45, -1e-45], (B, Hkv, S))
    acc = acc.astype(np.float32)
    pos = np.stack([[rng.permutation(S).astype(np.int32) - (5 if weights == "odd" else 0) for _ in range(Hkv)] for _ in range(B)])
    d_acc, d_pos = torch.from_numpy(acc).cuda(), torch.from_numpy(pos).cuda()
    d_lens = torch.tensor(lens, dtype=torch.int32).cuda()
    acc_out, pos_out = torch.full_like(d_acc, MARK), torch.full_like(d_pos, 7)
    src, lens_out = torch.full((B, Hkv, keep), 77, dtype=torch.int32, device="cuda"), torch.full((B,), 99, dtype=torch.int32, device="cuda")
    k1, v1 = k.clone(), v.clone()
    fr.fr_cache_evict(ptr(k1), ptr(v1), ptr(d_acc), ptr(d_pos), ptr(d_lens), ptr(acc_out), ptr(pos_out), ptr(lens_out),
                      ptr(src), B, Hkv, S, dh, fr.FR_DTYPE_F32 if dt == "f32" else fr.FR_DTYPE_BF16, keep, recent, stream())
    assert fr.fr_ops_sync_status(stream()) == 0
    assert lens_out.tolist() == [min(n, keep) for n in lens]
    wk, wv = k.clone(), v.clone()
    wacc, wpos, wsrc = np.full_like(acc, MARK), np.full_like(pos, 7), np.full((B, Hkv, keep), 77, np.int32)
    for b, n in enumerate(lens):
        for h in range(Hkv if n >= 0 else 0):
            at = R.evict_one(acc[b, h, :n], pos[b, h, :n], keep, recent)
            m = len(at)
            wsrc[b, h, :m], wsrc[b, h, m:] = at, -1
            wacc[b, h, :m], wpos[b, h, :m] = acc[b, h][at], pos[b, h][at]
            t = torch.from_numpy(at).cuda()
            wk[b, h, :m], wv[b, h, :m] = k[b, h][t], v[b, h][t]
    assert np.array_equal(src.cpu().numpy(), wsrc)
    assert np.array_equal(acc_out.cpu().numpy(), wacc, equal_nan=True) and np.array_equal(pos_out.cpu().numpy(), wpos)
    assert torch.equal(k1, wk) and torch.equal(v1, wv)
    assert torch.equal(d_acc.cpu(), torch.from_numpy(acc)) or weights == "odd"


def test_evict_refuses_bad_lengths_on_the_device():
    B, Hkv, S, dh, keep = 3, 2, 64, 64, 8
    k = torch.randn(B, Hkv, S, dh).cuda()
    k0, v = k.clone(), k.clone()
    acc, pos = torch.rand(B, Hkv, S).cuda(), torch.arange(S, dtype=torch.int32).expand(B, Hkv, S).contiguous().cuda()
    lens = torch.tensor([65, 8, 2 ** 30], dtype=torch.int32).cuda()
    outs = [torch.full_like(acc, MARK), torch.full_like(pos, 7), torch.zeros_like(lens), torch.full((B, Hkv, keep), 77, dtype=torch.int32).cuda()]
    fr.fr_cache_evict(ptr(k), ptr(v), ptr(acc), ptr(pos), ptr(lens), *[ptr(t) for t in outs], B, Hkv, S, dh, fr.FR_DTYPE_F32, keep, 2, stream())
    assert torch.equal(k, k0) and outs[2].tolist() == [65, 8, 2 ** 30]
    assert (outs[0][[0, 2]] == MARK).all() and (outs[3][[0, 2]] == 77).all() and outs[3][1, 0].tolist() == list(range(8))
    with pytest.raises(fr.FrError) as e:
        fr.fr_ops_sync_status(stream())
    assert e.value.code == fr.FR_ERR_DEVICE and "c001" in str(e.value)


@pytest.mark.parametrize("spec", [
    (4096, 2, 1, 64, 1, 40, [(7 * b) % 41 - 1 for b in range(4096)], "chain"),   # as many samples as there may be
    (1, 1024, 1, 64, 2, 300, [271], "tree"),                  # as many heads, one KV head: sixteen row tiles
    (2, 1024, 1024, 64, 1, 140, [139, 60], "chain"),
    (1, 64, 1, 64, 256, 400, [140], "tree"),                  # 128 row tiles: several batches
], ids=lambda s: "-".join(map(str, s[:6])) + "-" + s[7])
def test_attention_and_weights_at_their_limits(spec):
    c = Case(*spec).device()
    c.run()
    o = c.oracle()
    check(c, c.o, c.lse, o)
    acc = torch.zeros(c.B, c.Hkv, c.S, device="cuda")
    fr.fr_attention_weights(ptr(c.dq), ptr(c.dk), ptr(c.lse), ptr(c.dlens), ptr(c.dwords), 0, ptr(acc), c.B, c.Hq, c.Hkv, c.N, c.S,
                            c.dh, stream())
    lse = c.lse.double().cpu().numpy()
    want, w = R.weigh(c.q.double().numpy(), c.k.double().numpy(), lse, c.lens, c.words, None, np.zeros((c.B, c.Hkv, c.S)))
    tl = c.dh * 2.0 ** -24 * o[3].max() + (8 + np.abs(np.where(np.isinf(o[2]), 0.0, o[2])).max()) * 2.0 ** -21
    tol = w * (tl + c.Hq // c.Hkv * c.N * 2.0 ** -24) + 2.0 ** -23 * want + 1e-37
    for b, n in enumerate(c.lens):
        used = n + c.N if n >= 0 else 0
        assert np.all(np.abs(acc[b].cpu().numpy()[:, :used] - want[b, :, :used]) <= tol[b, :, :used])
        assert float(acc[b, :, used:].abs().sum()) == 0.0
    assert fr.fr_ops_sync_status(stream()) == 0


def test_bits_past_the_drafted_tokens_are_ignored():
    """In the last word of a mask row, of the tokens in use, and in a padded sample's words."""
    c = Case(3, 4, 2, 128, 37, 400, [300, -1, 5], "random").device()
    use = np.zeros((3, 2), np.uint32)
    use[:, 0], use[:, 1] = 0xF0F0F0F1, 0x15
    res = []
    for junk in (0, 0xFFFFFFE0):
        c.dwords[:, :, 1] |= int(np.uint32(junk).view(np.int32))
        c.dwords[1] = -1 if junk else 0
        d_use = torch.from_numpy((use | np.array([0, junk], np.uint32)).view(np.int32)).cuda()
        acc = torch.zeros(c.B, c.Hkv, c.S, device="cuda")
        c.run()
        fr.fr_attention_weights(ptr(c.dq), ptr(c.dk), ptr(c.lse), ptr(c.dlens), ptr(c.dwords), ptr(d_use), ptr(acc), c.B, c.Hq, c.Hkv,
                                c.N, c.S, c.dh, stream())
        res.append((c.o.clone(), c.lse.clone(), acc))
    assert all(torch.equal(x, y) for x, y in zip(*res))
    check(c, c.o, c.lse)


@pytest.mark.parametrize("B,Hkv", [(4096, 2), (2, 1024)])
def test_commit_and_evict_at_their_limits(B, Hkv):
    """As many samples and heads as there may be; equal positions, so that all slots are protected."""
    N, S, dh, keep, rng = 4, 12, 8, 5, np.random.default_rng(B)
    lens = rng.integers(-1, S - N + 1, B).astype(np.int32)
    npath = rng.integers(0, N + 1, B).astype(np.int32)
    path = np.stack([np.sort(rng.permutation(N)) for _ in range(B)]).astype(np.int32)
    for b in range(B):
        path[b, :npath[b]] = np.sort(rng.permutation(N)[:npath[b]])
    k = rng.standard_normal((B, Hkv, S, dh)).astype(np.float32)
    acc, pos = rng.random((B, Hkv, S)).astype(np.float32), np.where(np.arange(B) % 2, 9, np.arange(S)[:, None]).T[:, None].repeat(Hkv, 1)
    pos = np.ascontiguousarray(pos.astype(np.int32))
    dk, dv, dacc, dpos = (torch.from_numpy(x).cuda() for x in (k, -k, acc, pos))
    dl, dp, dn = (torch.from_numpy(x).cuda() for x in (lens, path, npath))
    l2, l3 = torch.full_like(dl, 99), torch.full_like(dl, 99)
    acc2, pos2, src = torch.full_like(dacc, MARK), torch.full_like(dpos, 7), torch.full((B, Hkv, keep), 77, dtype=torch.int32).cuda()
    fr.fr_cache_commit(ptr(dk), ptr(dv), ptr(dacc), ptr(dpos), ptr(dl), ptr(dp), ptr(dn), ptr(l2), B, Hkv, N, S, dh, fr.FR_DTYPE_F32,
                       stream())
    fr.fr_cache_evict(ptr(dk), ptr(dv), ptr(dacc), ptr(dpos), ptr(l2), ptr(acc2), ptr(pos2), ptr(l3), ptr(src), B, Hkv, S, dh,
                      fr.FR_DTYPE_F32, keep, 2, stream())
    assert fr.fr_ops_sync_status(stream()) == 0
    wk, wsrc = k.copy(), np.full((B, Hkv, keep), 77, np.int32)
    wacc, wpos = acc.copy(), pos.copy()
    racc, rpos = np.full_like(acc, MARK), np.full_like(pos, 7)
    for b, n in enumerate(lens):
        if n < 0:
            continue
        at, m = n + path[b, :npath[b]], n + npath[b]
        for x in (wk, wacc, wpos):
            x[b, :, n:m] = x[b][:, at]
        for h in range(Hkv):
            t = R.evict_one(wacc[b, h, :m], wpos[b, h, :m], keep, 2)
            wk[b, h, :len(t)] = wk[b, h][t]
            wsrc[b, h, :len(t)], wsrc[b, h, len(t):] = t, -1
            racc[b, h, :len(t)], rpos[b, h, :len(t)] = wacc[b, h][t], wpos[b, h][t]
    assert l2.tolist() == np.where(lens < 0, lens, lens + npath).tolist()
    assert l3.tolist() == np.where(lens < 0, lens, np.minimum(lens + npath, keep)).tolist()
    for got, want in ((dk, wk), (dv, -wk), (src, wsrc), (acc2, racc), (pos2, rpos)):
        assert np.array_equal(got.cpu().numpy(), want)


def test_pointers_of_the_host_are_refused():
    t = torch.zeros(4096, dtype=torch.bfloat16)
    d = torch.zeros(4096, dtype=torch.bfloat16, device="cuda")
    n = torch.zeros(4, dtype=torch.int32, device="cuda")
    for q, k, lens in ((t, d, n), (d, t, n), (d, d, torch.zeros(4, dtype=torch.int32))):
        with pytest.raises(fr.FrError) as e:
            fr.fr_attention_tree(ptr(q), ptr(k), ptr(d), ptr(lens), 0, ptr(d), 0, 1, 1, 1, 1, 8, 64, 0, 0, stream())
        assert e.value.code == fr.FR_ERR_ARG and "current device" in str(e.value)


class _Device:
    """A handle's device buffer as a torch tensor, without a copy."""

    def __init__(self, address, shape, typestr):
        self.__cuda_array_interface__ = {"data": (address, False), "shape": tuple(shape), "typestr": typestr, "version": 3}


def test_a_run_together_on_a_handles_cache():
    """Prefix pass, then two rounds on one layer of its KV cache: draft, attend, accept, weigh, commit, evict.
    Every step against its definition on the state that the step before left."""
    import synthetic
    cfg = synthetic.PrefixConfig("run", L=2, D=256, Hq=4, Hkv=2, dh=64, F=512, B=2, P=150, dtype="bf16")
    inp = synthetic.make_prefix_pass_inputs(cfg, seed=4)
    room = 230                                     # the handle's largest prefix: room behind this one's 150 tokens
    backbone = fr.PrefixPass(cfg, P_max=room)
    backbone.load_weights(inp["weights"])
    backbone.run(torch.from_numpy(inp["emb"]).bfloat16().cuda())
    assert backbone.sync_status() == 0
    address_k, nbytes = backbone.buffer("kv_k")
    address_v, _ = backbone.buffer("kv_v")
    layer_bytes = nbytes // cfg.L
    S = room + 1                                   # slots per (sample, KV head) of this handle
    assert layer_bytes // (cfg.B * cfg.Hkv * cfg.dh * 2) == S
    shape, layer = (cfg.B, cfg.Hkv, S, cfg.dh), 1
    k = torch.as_tensor(_Device(address_k + layer * layer_bytes, shape, "<i2"), device="cuda").view(torch.bfloat16)
    v = torch.as_tensor(_Device(address_v + layer * layer_bytes, shape, "<i2"), device="cuda").view(torch.bfloat16)
    assert k.data_ptr() == address_k + layer * layer_bytes
    got_k, _ = backbone.read_kv(layer, 1, 150)
    assert np.array_equal(k[1, :, :150].contiguous().view(torch.int16).cpu().numpy().view(np.uint16), got_k)

    rng, g = np.random.default_rng(0), torch.Generator().manual_seed(0)
    B, Hq, Hkv, dh, N, keep, recent = cfg.B, cfg.Hq, cfg.Hkv, cfg.dh, 13, 120, 16
    acc, acc2 = torch.zeros(B, Hkv, S).cuda(), torch.zeros(B, Hkv, S).cuda()
    pos = torch.arange(S, dtype=torch.int32).expand(B, Hkv, S).contiguous().cuda()
    pos2 = torch.zeros_like(pos)
    lens, lens2 = torch.tensor([150, 150], dtype=torch.int32).cuda(), torch.zeros(2, dtype=torch.int32).cuda()
    src = torch.zeros(B, Hkv, keep, dtype=torch.int32).cuda()
    for step in range(2):
        n = lens.tolist()
        words = np.stack([fr.fr_tree_mask([int(rng.integers(-1, i)) if i else -1 for i in range(N)]) for _ in range(B)])
        d_words = torch.from_numpy(words.view(np.int32)).cuda()
        for b in range(B):   # the drafts' rows and positions
            k[b, :, n[b]:n[b] + N] = torch.randn(Hkv, N, dh, generator=g).bfloat16().cuda()
            v[b, :, n[b]:n[b] + N] = torch.randn(Hkv, N, dh, generator=g).bfloat16().cuda()
            pos[b, :, n[b]:n[b] + N] = 1000 * (step + 1) + torch.arange(N, dtype=torch.int32).cuda()
        c = Case.__new__(Case)
        c.B, c.Hq, c.Hkv, c.dh, c.N, c.S, c.lens, c.words = B, Hq, Hkv, dh, N, S, n, words
        c.q = (torch.randn(B, Hq, N, dh, generator=g) * 1.5).bfloat16()
        c.k, c.v = k.cpu(), v.cpu()
        c.device()
        fr.fr_attention_tree(ptr(c.dq), ptr(k), ptr(v), ptr(lens), ptr(d_words), ptr(c.o), ptr(c.lse), B, Hq, Hkv, N, S, dh,
                             ptr(c.scratch), c.nscratch, stream())
        oracle = c.oracle()
        check(c, c.o, c.lse, oracle)

        path = np.zeros((B, N), np.int32)   # the accepted branch: the deepest token's ancestors
        npath = np.zeros(B, np.int32)
        use = np.zeros((B, 1), np.uint32)
        for b in range(B):
            best = max(range(N), key=lambda i: bin(int(words[b, i, 0])).count("1"))
            nodes = [j for j in range(N) if (int(words[b, best, 0]) >> j) & 1]
            npath[b] = len(nodes)
            path[b, :len(nodes)] = nodes
            use[b, 0] = words[b, best, 0]
        d_use, d_path, d_np = (torch.from_numpy(x).cuda() for x in (use.view(np.int32), path, npath))
        before, lse = acc.cpu().numpy(), c.lse.double().cpu().numpy()
        fr.fr_attention_weights(ptr(c.dq), ptr(k), ptr(c.lse), ptr(lens), ptr(d_words), ptr(d_use), ptr(acc), B, Hq, Hkv, N, S,
                                dh, stream())
        want, _ = R.weigh(c.q.double().numpy(), c.k.double().numpy(), lse, n, words, use, before)
        for b in range(B):
            m = n[b] + N
            assert np.all(np.abs(acc[b, :, :m].cpu().numpy() - want[b, :, :m]) <= 2.0 ** -13 * want[b, :, :m] + 1e-30)

        fr.fr_cache_commit(ptr(k), ptr(v), ptr(acc), ptr(pos), ptr(lens), ptr(d_path), ptr(d_np), ptr(lens2), B, Hkv, N, S, dh,
                           fr.FR_DTYPE_BF16, stream())
        lens, lens2 = lens2, lens
        assert lens.tolist() == [x + int(y) for x, y in zip(n, npath)]
        for b in range(B):
            at = torch.from_numpy(n[b] + path[b, :npath[b]].astype(np.int64))
            assert torch.equal(k[b, :, n[b]:n[b] + npath[b]].cpu(), c.k[b][:, at])
        state = [x.clone() for x in (k, v, acc, pos)]
        fr.fr_cache_evict(ptr(k), ptr(v), ptr(acc), ptr(pos), ptr(lens), ptr(acc2), ptr(pos2), ptr(lens2), ptr(src), B, Hkv, S,
                          dh, fr.FR_DTYPE_BF16, keep, recent, stream())
        m = lens.tolist()
        assert lens2.tolist() == [min(x, keep) for x in m]
        for b in range(B):
            for h in range(Hkv):
                at = R.evict_one(state[2][b, h, :m[b]].cpu().numpy(), state[3][b, h, :m[b]].cpu().numpy(), keep, recent)
                t = torch.from_numpy(at).cuda()
                assert src[b, h, :len(at)].tolist() == at.tolist()
                for new, old in zip((k, v, acc2, pos2), state):
                    assert torch.equal(new[b, h, :len(at)], old[b, h][t])
        acc, acc2, pos, pos2, lens, lens2 = acc2, acc, pos2, pos, lens2, lens
    assert fr.fr_ops_sync_status(stream()) == 0
    backbone.close()


def weigh_on_the_gpu(c, lse, acc):
    """R.weigh on the GPU in 64 bits, all tokens in use: for caches too long for the numpy loops."""
    out, weight, g = acc.double().clone(), torch.zeros_like(acc, dtype=torch.float64), c.Hq // c.Hkv
    for b, n in enumerate(c.lens):
        if n < 0:
            continue
        hidden = torch.from_numpy(~R.sees(None if c.words is None else c.words[b], c.N)).cuda()
        for h in range(c.Hq):
            x = c.dq[b, h].double() @ c.dk[b, h // g, :n + c.N].double().T / c.dh ** 0.5 - lse[b, h].double()[:, None]
            x[:, n:][hidden] = float("-inf")
            weight[b, h // g, :n + c.N] += torch.where((lse[b, h] == float("-inf"))[:, None], 0.0, torch.exp(x)).sum(0)
        out[b, :, :n] += weight[b, :, :n]
        out[b, :, n:n + c.N] = weight[b, :, n:n + c.N]
    return out, weight


# rows of a KV head past 256 are summed in several passes: two with one, two and many tiles per CTA, three, eight,
# 64; blocks of tiles within a CTA's share (the last)
MANY_ROWS = [(1, 8, 1, 256, 63, 300, [200], "tree"), (6, 8, 1, 256, 63, 9000, [8900, 7000, 8555, 130, -1, 0], "tree"),
             (2, 6, 2, 128, 130, 2300, [2100, 1999], "chain"), (7, 3, 1, 64, 256, 40000, [39000 + 31 * b for b in range(7)], "tree"),
             (3, 8, 1, 128, 256, 6000, [5700, 3333, 40], "tree"), (1, 64, 1, 64, 256, 400, [140], "tree"),
             (8, 6, 2, 64, 100, 160000, [159900 - 7 * b for b in range(8)], "tree")]


@pytest.mark.parametrize("spec", MANY_ROWS, ids=lambda s: "-".join(map(str, s[:6])) + "-" + s[7])
def test_weights_of_many_rows_are_added_to_large_sums_at_once(spec):
    """A slot's sum over all rows is one float32 value, added with one rounding: half a step of the result, 2^-24,
    beside the error of the sum itself."""
    c = Case(*spec)
    rows = c.Hq // c.Hkv * c.N
    assert rows > 256
    c.device().run()
    acc = (500 + 1500 * torch.rand(c.B, c.Hkv, c.S, generator=torch.Generator().manual_seed(1))).cuda()
    want, w = weigh_on_the_gpu(c, c.lse, acc)
    got = [acc.clone() for _ in range(2)]
    for x in got:
        fr.fr_attention_weights(ptr(c.dq), ptr(c.dk), ptr(c.lse), ptr(c.dlens), ptr(c.dwords), 0, ptr(x), c.B, c.Hq, c.Hkv, c.N, c.S,
                                c.dh, stream())
    assert torch.equal(*got) and fr.fr_ops_sync_status(stream()) == 0
    # |q| |k| bounds sum|q_d k_d|; |lse| is at most the largest score and the log of the slots
    live = [b for b, n in enumerate(c.lens) if n >= 0]
    size = max(float((c.dq[b].float().norm(dim=-1).max() * c.dk[b, :, :c.lens[b] + c.N].float().norm(dim=-1).max())) for b in live) / c.dh ** 0.5
    tl = c.dh * 2.0 ** -24 * size + (8 + size + np.log(c.S)) * 2.0 ** -21
    for b, n in enumerate(c.lens):
        m = n + c.N if n >= 0 else 0
        d = (got[0][b].double() - want[b]).abs()
        assert torch.all(d[:, :m] <= w[b, :, :m] * (tl + rows * 2.0 ** -24) + 2.0 ** -24 * want[b, :, :m] + 1e-37), float(d[:, :m].max())
        assert torch.equal(got[0][b, :, m:], acc[b, :, m:])


# a cluster per unit (one and several samples), units whole, cut units that the merge joins, several row tiles, batches of them
GIVE_UP = [(1, 8, 1, 256, 1, 866, [816], "chain"), (2, 16, 16, 64, 128, 4300, [4095, 3900], "chain"), (4, 16, 2, 128, 24, 2148, [2048, 1500, -1, 9], "tree"),
           (40, 8, 8, 64, 1, 200, [150 + b for b in range(40)], "chain"), (24, 32, 8, 128, 1, 4200, [4190 - 97 * b for b in range(24)], "chain"),
           (6, 8, 1, 256, 63, 9000, [8900 - 500 * b for b in range(6)], "tree"), (2, 34, 1, 64, 64, 6000, [5900, 3333], "chain")]


@pytest.mark.parametrize("spec", GIVE_UP, ids=lambda s: "-".join(map(str, s[:6])))
def test_a_wait_that_gives_up_leaves_what_it_has_not_computed(spec):
    """At 1 ns every CTA's first wait gives up, and nothing is written; at a few microseconds some of them do, and
    what is written is right.  The call says so, and the next one is whole again."""
    c = Case(*spec).device()
    c.run()
    o, lse = c.o.clone(), c.lse.clone()
    acc0 = torch.rand(c.B, c.Hkv, c.S, generator=torch.Generator().manual_seed(2)).cuda()

    def weights():
        acc = acc0.clone()
        fr.fr_attention_weights(ptr(c.dq), ptr(c.dk), ptr(lse), ptr(c.dlens), ptr(c.dwords), 0, ptr(acc), c.B, c.Hq, c.Hkv, c.N, c.S,
                                c.dh, stream())
        return acc

    acc = weights()
    assert fr.fr_ops_sync_status(stream()) == 0

    def gave_up(codes):
        try:
            return fr.fr_ops_sync_status(stream())
        except fr.FrError as e:
            assert e.code == fr.FR_ERR_TIMEOUT and any(f"0x{x:08x}" in str(e) for x in codes), e
            return e.code

    marks = torch.full_like(o, MARK), torch.full_like(lse, MARK)
    try:
        for limit in (1, 300, 1000, 2000, 4000, 8000, 16000, 1):
            fr.fr_ops_set_wait_limit(limit)
            c.o.fill_(MARK), c.lse.fill_(MARK)
            c.run()
            rc = gave_up((0x710, 0x711, 0x713))
            if limit == 1:
                assert rc == fr.FR_ERR_TIMEOUT and torch.equal(c.o, marks[0]) and torch.equal(c.lse, marks[1])
            elif rc == 0:
                assert torch.equal(c.o, o) and torch.equal(c.lse, lse)
            assert bool(((c.o == o) | (c.o == MARK)).all()) and bool(((c.lse == lse) | (c.lse == MARK)).all())
            got = weights()
            rc = gave_up((0x720, 0x721, 0x723))
            if limit == 1:
                assert rc == fr.FR_ERR_TIMEOUT and torch.equal(got, acc0)
            elif rc == 0:
                assert torch.equal(got, acc)
            assert bool(((got == acc) | (got == acc0)).all())
    finally:
        fr.fr_ops_set_wait_limit(0)
    c.run()
    assert torch.equal(c.o, o) and torch.equal(c.lse, lse) and torch.equal(weights(), acc)
    assert fr.fr_ops_sync_status(stream()) == 0


@pytest.mark.parametrize("spec", [
    (8, 8, 1, 256, 5, 4000, [3900, 3, -1, 0, 60, -1, 7, 100], "tree"),                 # a cluster per unit
    (9, 8, 1, 128, 1, 8300, [-1, 0, 1, 127, 8299, -1, 128, 2, 30], "chain"),
    (74, 4, 1, 64, 3, 4100, [(b * 5) % 90 - 1 if b != 40 else 4097 for b in range(74)], "tree"),
    (74, 4, 1, 64, 3, 12000, [(b * 5) % 90 - 1 if b != 73 else 11990 for b in range(74)], "tree"),   # more tiles than a cluster takes
], ids=lambda s: "-".join(map(str, s[:6])))
def test_one_long_sample_among_short_and_padded_ones(spec):
    c = Case(*spec).device()
    c.run()
    o = c.oracle()
    check(c, c.o, c.lse, o)
    acc = torch.zeros(c.B, c.Hkv, c.S, device="cuda")
    c.lse[torch.tensor(c.lens) < 0] = float("-inf")
    fr.fr_attention_weights(ptr(c.dq), ptr(c.dk), ptr(c.lse), ptr(c.dlens), ptr(c.dwords), 0, ptr(acc), c.B, c.Hq, c.Hkv, c.N, c.S,
                            c.dh, stream())
    want, w = R.weigh(c.q.double().numpy(), c.k.double().numpy(), c.lse.double().cpu().numpy(), c.lens, c.words, None, np.zeros(acc.shape))
    tl = c.dh * 2.0 ** -24 * o[3].max() + (8 + np.abs(np.where(np.isinf(o[2]), 0.0, o[2])).max()) * 2.0 ** -21
    for b, n in enumerate(c.lens):
        m = n + c.N if n >= 0 else 0
        d = np.abs(acc[b, :, :m].cpu().numpy() - want[b, :, :m])
        assert np.all(d <= w[b, :, :m] * (tl + c.Hq // c.Hkv * c.N * 2.0 ** -24) + 2.0 ** -24 * want[b, :, :m] + 1e-37)
        assert float(acc[b, :, m:].abs().sum()) == 0.0
    assert fr.fr_ops_sync_status(stream()) == 0


@pytest.mark.parametrize("S,keep,recent,dtype", [(70, 10, 3, torch.float32), (3000, 1100, 0, torch.bfloat16), (9000, 9000, 64, torch.float32)])
def test_evict_leaves_its_inputs_as_they_were(S, keep, recent, dtype):
    """Bit for bit, NaN and zeros of both signs among the sums; sums and positions that stay keep their bits too."""
    B, Hkv, dh, rng = 3, 2, 16, np.random.default_rng(S)
    bits = rng.choice(np.array([0, 0x80000000, 0x7fc00000, 0xffc01234, 0x7f800000, 0xff800000, 1, 0x80000001, 0x3f800000], np.uint32), (B, Hkv, S))
    acc, pos = torch.from_numpy(bits.view(np.float32)).cuda(), torch.from_numpy(rng.permutation(B * Hkv * S).astype(np.int32).reshape(B, Hkv, S)).cuda()
    lens = torch.tensor([S, -1, S // 2], dtype=torch.int32).cuda()
    k = torch.randn(B, Hkv, S, dh).to(dtype).cuda()
    v, ins = k.clone(), [x.clone() for x in (acc.view(torch.int32), pos, lens)]
    acc2, pos2, lens2 = torch.zeros_like(acc), torch.zeros_like(pos), torch.zeros_like(lens)
    src = torch.zeros(B, Hkv, keep, dtype=torch.int32).cuda()
    fr.fr_cache_evict(ptr(k), ptr(v), ptr(acc), ptr(pos), ptr(lens), ptr(acc2), ptr(pos2), ptr(lens2), ptr(src), B, Hkv, S, dh,
                      fr.FR_DTYPE_F32 if dtype == torch.float32 else fr.FR_DTYPE_BF16, keep, recent, stream())
    assert fr.fr_ops_sync_status(stream()) == 0
    for x, y in zip((acc.view(torch.int32), pos, lens), ins):
        assert torch.equal(x, y)
    for b in (0, 2):
        m = int(lens2[b])
        for h in range(Hkv):
            at = src[b, h, :m].long()
            assert torch.equal(acc2[b, h, :m].view(torch.int32), ins[0][b, h][at]) and torch.equal(pos2[b, h, :m], ins[1][b, h][at])


# one pass of rows, and several
@pytest.mark.parametrize("spec", [(5, 4, 2, 64, 3, 100, [50, 97, 20, 4, -1], "tree"), (4, 8, 1, 256, 63, 700, [637, 100, 50, 0], "tree"),
                                  (40, 8, 8, 128, 4, 300, [7 * b for b in range(40)], "chain")], ids=lambda s: "-".join(map(str, s[:6])))
def test_attention_weights_refuse_bad_lengths_on_the_device(spec):
    """lens + N past the cache, up to the largest int: those samples' sums stay as they were, the others' are right."""
    c = Case(*spec).device()
    c.run()
    acc0 = torch.rand(c.B, c.Hkv, c.S, generator=torch.Generator().manual_seed(3)).cuda()

    def weights():
        acc = acc0.clone()
        fr.fr_attention_weights(ptr(c.dq), ptr(c.dk), ptr(c.lse), ptr(c.dlens), ptr(c.dwords), 0, ptr(acc), c.B, c.Hq, c.Hkv, c.N, c.S,
                                c.dh, stream())
        return acc

    want = weights()
    assert fr.fr_ops_sync_status(stream()) == 0
    bad = [0, 2, c.B - 2]
    for b, n in zip(bad, (c.S - c.N + 1, 2 ** 31 - 1, c.S)):
        c.dlens[b] = n
        want[b] = acc0[b]
    got = weights()
    with pytest.raises(fr.FrError) as e:
        fr.fr_ops_sync_status(stream())
    assert e.value.code == fr.FR_ERR_DEVICE and "c001" in str(e.value)
    assert torch.equal(got, want) and fr.fr_ops_sync_status(stream()) == 0


# a cluster per unit, units whole, units cut between CTAs
@pytest.mark.parametrize("spec", [(2, 8, 1, 256, 7, 3000, [2900, 2500]), (40, 8, 8, 64, 2, 200, [150 + b % 40 for b in range(40)]),
                                  (24, 16, 8, 128, 3, 4200, [4190 - 97 * b for b in range(24)])], ids=lambda s: "-".join(map(str, s[:6])))
def test_committed_rows_that_are_not_finite(spec):
    """Values reach the features that hold them, of the rows of their KV head; a NaN or infinite score, its whole row."""
    c = Case(*spec, "tree").device()
    c.run()
    o, lse = c.o.clone().view(c.B, c.N, c.Hq, c.dh), c.lse.clone()
    g, b, h = c.Hq // c.Hkv, c.B - 1, c.Hkv - 1
    rows = slice(h * g, (h + 1) * g)
    c.dv[b, h, c.lens[b] // 2, 5], c.dv[b, h, 0, 33], c.dv[b, h, c.lens[b] - 1, 60] = float("nan"), float("inf"), float("-inf")
    c.run()
    o2 = c.o.clone().view(o.shape)
    assert not torch.isfinite(o2[b, :, rows][..., [5, 33, 60]]).any()
    for f in (5, 33, 60):
        o2[b, :, rows, f] = o[b, :, rows, f]
    assert torch.equal(o2, o) and torch.equal(c.lse, lse)
    c.dv.copy_(c.v)
    c.dk[b, h, c.lens[b] // 3, 2] = float("nan")
    c.run()
    o2 = c.o.clone().view(o.shape)
    assert torch.isnan(o2[b, :, rows]).all() and torch.isnan(c.lse[b, rows]).all()
    o2[b, :, rows] = o[b, :, rows]
    c.lse[b, rows] = lse[b, rows]
    assert torch.equal(o2, o) and torch.equal(c.lse, lse)
    assert fr.fr_ops_sync_status(stream()) == 0


def test_weights_of_many_rows_in_a_graph_and_on_two_streams():
    """Several passes of rows: a captured call follows the lengths; two calls that overlap in time do not share anything."""
    a, b = Case(3, 8, 1, 128, 90, 5000, [4900, 17, 4000], "tree").device(), Case(3, 8, 1, 128, 90, 5000, [1000, 4910, -1], "tree", seed=4).device()
    a.run(), b.run()
    acc0 = torch.rand(3, 1, 5000).cuda() * 100

    def weights(c, acc):
        fr.fr_attention_weights(ptr(c.dq), ptr(c.dk), ptr(c.lse), ptr(c.dlens), ptr(c.dwords), 0, ptr(acc), 3, 8, 1, 90, 5000, 128,
                                torch.cuda.current_stream().cuda_stream)

    want = [acc0.clone(), acc0.clone()]
    weights(a, want[0]), weights(b, want[1])
    assert not torch.equal(*want)
    got, s = [acc0.clone(), acc0.clone()], [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for c, x, st in zip((a, b), got, s):
        with torch.cuda.stream(st):
            for _ in range(4):
                x.copy_(acc0)
                weights(c, x)
    torch.cuda.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    acc, graph = acc0.clone(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s[0]):
        weights(a, acc)
    graph.replay()
    assert torch.equal(acc, want[0])
    for x, y in ((a.dq, b.dq), (a.dk, b.dk), (a.lse, b.lse), (a.dlens, b.dlens), (a.dwords, b.dwords), (acc, acc0)):
        x.copy_(y)
    graph.replay()
    assert torch.equal(acc, want[1]) and fr.fr_ops_sync_status(stream()) == 0

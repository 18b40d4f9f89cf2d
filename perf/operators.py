"""Operators on the static KV cache: tree attention, accumulated attention weights, commit of accepted
drafts, eviction by accumulated weight.

The cache of a layer is K and V [B][Hkv][S_max][dh]; sample b holds lens[b] committed tokens in slots
0..lens[b]-1 and, while drafts are being verified, N drafted tokens in slots lens[b]..lens[b]+N-1.
lens[b] < 0 marks a padded sample of the batch: it is skipped and all its data stays as it was.

  attend   o = softmax(q k^T / sqrt(dh)) v of N drafted tokens over the committed slots and, by a bit mask
           per token, the drafted ones (a tree: its ancestors and itself), with the log-sum-exp of each row
  weigh    acc[b][hkv][s] += the attention weight slot s received from the rows in use (heads of the KV
           head's group x drafted tokens); the drafted slots' acc is set
  commit   the slots of the accepted drafted tokens move down to follow the committed ones
  evict    the `keep` slots of largest acc stay, the `recent` last positions before all others; kept slots
           at or past `keep` move into the freed slots below it, both in ascending order
"""
import math

import numpy as np
import torch

own = False   # False: the plain forms below; True: the framework's kernels

INACTIVE = -1


def listed():
    return [
        # one token of the action policy's backbone over one observation's prefix: latency
        dict(name="attend_n1_b1", op="attend", B=1, Hq=8, Hkv=1, dh=256, N=1, S_max=866, len=816, ragged=0.0, pad=0, mask="chain"),
        # small trees for a few robots at the stress shape's heads, ragged histories, one padded sample
        dict(name="attend_n24_b4", op="attend", B=4, Hq=16, Hkv=2, dh=128, N=24, S_max=2148, len=2048, ragged=0.3, pad=1, mask="tree"),
        # single-token decode of a large batch over long ragged caches: streams the cache
        dict(name="attend_n1_b32", op="attend", B=32, Hq=32, Hkv=8, dh=128, N=1, S_max=8200, len=8191, ragged=0.8, pad=0, mask="chain"),
        # a 63-node tree over a long cache, one KV head for eight query heads: arithmetic
        dict(name="attend_n63_b6", op="attend", B=6, Hq=8, Hkv=1, dh=256, N=63, S_max=33000, len=32767, ragged=0.1, pad=0, mask="tree"),
        # a chunk of 128 tokens in sequence without shared heads
        dict(name="attend_n128_b2", op="attend", B=2, Hq=16, Hkv=16, dh=64, N=128, S_max=4300, len=4095, ragged=0.05, pad=0, mask="chain"),
        # the weights of the same calls: a single token, a large batch, a tree with part of its tokens accepted
        dict(name="weigh_n1_b1", op="weigh", B=1, Hq=8, Hkv=1, dh=256, N=1, S_max=866, len=816, ragged=0.0, pad=0, mask="chain"),
        dict(name="weigh_n1_b32", op="weigh", B=32, Hq=32, Hkv=8, dh=128, N=1, S_max=8200, len=8191, ragged=0.8, pad=0, mask="chain"),
        dict(name="weigh_n63_b6", op="weigh", B=6, Hq=8, Hkv=1, dh=256, N=63, S_max=33000, len=32767, ragged=0.1, pad=0, mask="tree"),
        # accepted tokens of one robot's draft, and of a large batch's
        dict(name="commit_n24_b1", op="commit", B=1, Hkv=1, dh=256, N=24, S_max=866, len=816, ragged=0.0, pad=0, dtype="float32"),
        dict(name="commit_n63_b64", op="commit", B=64, Hkv=8, dh=128, N=63, S_max=2148, len=2048, ragged=0.3, pad=3, dtype="bfloat16"),
        # pruning one observation's prefix to its most attended tokens; trimming a batch of long histories
        dict(name="evict_b1", op="evict", B=1, Hkv=1, dh=256, S_max=866, len=866, ragged=0.0, pad=0, keep=512, recent=50, dtype="bfloat16"),
        dict(name="evict_b16", op="evict", B=16, Hkv=8, dh=128, S_max=16500, len=16384, ragged=0.2, pad=1, keep=12001, recent=256, dtype="bfloat16"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attend", "attend", "weigh", "commit", "evict"])
    dh = rng.choice([64, 128, 256])
    group, Hkv = rng.choice([(8, 1), (8, 2), (4, 8), (1, 16), (1, 4), (7, 1), (3, 2), (16, 1)])
    ragged, dtype = rng.choice([0.0, 0.1, 0.5, 0.9]), rng.choice(["bfloat16", "bfloat16", "float32"])
    length = _log_int(rng, 1, 33000)
    B = _log_int(rng, 1, 64)
    room = rng.randrange(0, 100)
    if op in ("attend", "weigh"):
        N = _log_int(rng, 1, 256)
        S = length + N + room
        # no more cache and no more arithmetic than the largest listed cases
        while B > 1 and (B * Hkv * S * dh > 1.6e8 or B * Hkv * group * N * S * dh > 2.4e10):
            B //= 2
        while N > 1 and Hkv * group * N * S * dh > 2.4e10:
            N //= 2
        return dict(op=op, B=B, Hq=group * Hkv, Hkv=Hkv, dh=dh, N=N, S_max=length + N + room, len=length, ragged=ragged,
                    pad=rng.choice([0, 0, 1]) if B > 1 else 0, mask=rng.choice(["tree", "chain"]))
    N = _log_int(rng, 1, 128)
    length = max(length, 2)
    S = length + N + room
    while B > 1 and B * Hkv * S * dh > (0.8e8 if dtype == "float32" else 1.6e8):
        B //= 2
    pad = rng.choice([0, 0, 1]) if B > 1 else 0
    if op == "commit":
        return dict(op=op, B=B, Hkv=Hkv, dh=dh, N=N, S_max=S, len=length, ragged=ragged, pad=pad, dtype=dtype)
    keep = max(1, int(length * rng.uniform(0.1, 1.0)))
    return dict(op=op, B=B, Hkv=Hkv, dh=dh, S_max=S, len=length, ragged=ragged, pad=pad, keep=keep,
                recent=rng.randrange(0, keep + 1) if rng.random() < 0.5 else min(keep, 32), dtype=dtype)


def _lens(case):
    """Committed tokens of each sample: spread below case['len'], padded samples last."""
    B = case["B"]
    out = [case["len"] - int(case["ragged"] * case["len"] * ((b * 0.6180339887) % 1.0)) for b in range(B)]
    for b in range(B - case["pad"], B):
        out[b] = INACTIVE
    return out


def _tree_words(rng, B, N, kind):
    """Mask words [B][N][ceil(N/32)]: a token sees itself and its ancestors."""
    vis = np.zeros((B, N, N), np.uint8)
    bi = np.arange(B)
    for i in range(N):
        if i:
            # a parent among the 8 tokens before it, or the root (the committed tokens alone)
            back = rng.integers(1, 9, B) if kind == "tree" else np.ones(B, np.int64)
            parent = i - back
            vis[bi, i] = np.where((parent >= 0)[:, None], vis[bi, np.maximum(parent, 0)], 0)
        vis[:, i, i] = 1
    W = (N + 31) // 32
    bits = np.zeros((B, N, W * 32), np.uint8)
    bits[:, :, :N] = vis
    return np.packbits(bits, axis=-1, bitorder="little").view("<u4").astype(np.uint32).view(np.int32).reshape(B, N, W)


def _rows(gen, shape, dtype):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32 if dtype == "float32" else torch.bfloat16)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rng = np.random.default_rng(seed)
    op, B, Hkv, dh, S = case["op"], case["B"], case["Hkv"], case["dh"], case["S_max"]
    lens = _lens(case)
    st = dict(case, lens_host=lens, lens=torch.tensor(lens, dtype=torch.int32, device="cuda"))
    st["k"] = _rows(gen, (B, Hkv, S, dh), case.get("dtype", "bfloat16"))
    if op in ("attend", "weigh"):
        N, Hq = case["N"], case["Hq"]
        st["q"] = (torch.randn((B, Hq, N, dh), generator=gen, device="cuda") * 1.5).to(torch.bfloat16)
        st["words"] = torch.from_numpy(_tree_words(rng, B, N, case["mask"])).cuda()
        if case["mask"] == "chain":
            st["words"] = None   # the operators' own default: a sequence, each token sees those before it
    if op == "attend":
        st["v"] = _rows(gen, (B, Hkv, S, dh), "bfloat16")
        st["o"] = torch.zeros(B, N, Hq * dh, dtype=torch.bfloat16, device="cuda")
        st["lse"] = torch.zeros(B, Hq, N, device="cuda")
        # a workspace that the program keeps: 40 MiB cover every size
        st["scratch"] = torch.empty(40 << 20, dtype=torch.uint8, device="cuda")
    elif op == "weigh":
        # the log-sum-exp that the attention call left, the sums so far, and the tokens that were accepted
        st["lse"] = _weigh_lse(st)
        st["acc"] = torch.rand((B, Hkv, S), generator=gen, device="cuda")
        st["use"] = None
        if case["mask"] == "tree":
            bits = (rng.random((B, N)) < 0.5).astype(np.uint8)
            words = np.packbits(np.pad(bits, ((0, 0), (0, -N % 32))), axis=-1, bitorder="little").view("<u4")
            st["use"] = torch.from_numpy(words.astype(np.uint32).view(np.int32).reshape(B, -1)).cuda()
    else:
        st["v"] = _rows(gen, (B, Hkv, S, dh), case["dtype"])
        # weights fall off over two decades, as summed attention does
        st["acc"] = torch.exp(torch.randn((B, Hkv, S), generator=gen, device="cuda") * 1.5)
        st["pos"] = torch.argsort(torch.rand((B, Hkv, S), generator=gen, device="cuda"), dim=-1).to(torch.int32)
        st["lens_out"] = torch.zeros(B, dtype=torch.int32, device="cuda")
        if op == "commit":
            N = case["N"]
            npath = rng.integers(0, N + 1, B)
            path = np.zeros((B, N), np.int32)
            for b in range(B):
                path[b, :npath[b]] = np.sort(rng.permutation(N)[:npath[b]])
            st["path"] = torch.from_numpy(path).cuda()
            st["npath"] = torch.from_numpy(npath.astype(np.int32)).cuda()
        else:
            st["acc_out"] = torch.zeros_like(st["acc"])
            st["pos_out"] = torch.zeros_like(st["pos"])
            st["src"] = torch.zeros(B, Hkv, case["keep"], dtype=torch.int32, device="cuda")
    return st


# ------------------------------------------------------------------ plain forms

def _visible(st, S):
    """[B][N][S] truth values: slot s counts for drafted token n of sample b."""
    B, N = st["B"], st["N"]
    dev = st["lens"].device
    slot = torch.arange(S, device=dev)
    j = slot[None, :] - st["lens"][:, None].long()                        # [B][S] drafted index, < 0: committed
    if st["words"] is None:
        drafted = torch.arange(N, device=dev)[None, :, None] >= j[:, None, :]
    else:
        jc = j.clamp(0, N - 1)
        word = torch.gather(st["words"].long(), 2, (jc // 32)[:, None, :].expand(B, N, S))
        drafted = ((word >> (jc % 32)[:, None, :]) & 1) == 1
    return ((j < 0)[:, None, :] | (drafted & (j < N)[:, None, :])) & (st["lens"] >= 0)[:, None, None]


def _scores(st, S):
    B, Hq, Hkv, N, dh = st["B"], st["Hq"], st["Hkv"], st["N"], st["dh"]
    g = Hq // Hkv
    q = st["q"].float().reshape(B, Hkv, g * N, dh)
    s = torch.matmul(q, st["k"][:, :, :S].float().transpose(2, 3)) * (1.0 / math.sqrt(dh))
    return s.reshape(B, Hkv, g, N, S).masked_fill(~_visible(st, S)[:, None, None], float("-inf"))


def _span(st):
    return max(1, max(st["lens_host"]) + st["N"])


def _weigh_lse(st):
    return torch.logsumexp(_scores(st, _span(st)), dim=-1).reshape(st["B"], st["Hq"], st["N"])


def _attend(st):
    B, Hq, Hkv, N, dh = st["B"], st["Hq"], st["Hkv"], st["N"], st["dh"]
    S = _span(st)
    s = _scores(st, S)
    m = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(torch.isinf(m), torch.zeros_like(m), m))
    l = p.sum(-1, keepdim=True)
    # slots past the drafted tokens hold whatever was there before
    used = torch.arange(S, device=s.device)[None, :] < st["lens"][:, None] + N
    v = st["v"][:, :, :S].float().masked_fill(~used[:, None, :, None], 0.0)
    o = torch.matmul((p / torch.where(l > 0, l, torch.ones_like(l))).reshape(B, Hkv, -1, S), v)
    o = o.reshape(B, Hq, N, dh).transpose(1, 2).reshape(B, N, Hq * dh).to(torch.bfloat16)
    active = (st["lens"] >= 0)[:, None, None]
    st["o"].copy_(torch.where(active, o, st["o"]))
    lse = (torch.log(l) + m).reshape(B, Hq, N)
    st["lse"].copy_(torch.where(active, lse, st["lse"]))
    return {"o": st["o"], "lse": st["lse"]}


def _weigh(st):
    B, Hq, Hkv, N = st["B"], st["Hq"], st["Hkv"], st["N"]
    S = _span(st)
    p = torch.exp(_scores(st, S) - st["lse"].reshape(B, Hkv, Hq // Hkv, N, 1))
    # a row that sees nothing has no weight to give
    p = p.masked_fill(~_visible(st, S)[:, None, None], 0.0)
    if st["use"] is not None:
        n = torch.arange(N, device=p.device)
        p = p * (((st["use"].long()[:, n // 32] >> (n % 32)) & 1) == 1).float()[:, None, None, :, None]
    w = p.sum((2, 3))
    slot, lens = torch.arange(S, device=p.device)[None, None], st["lens"][:, None, None]
    acc = st["acc"][:, :, :S]
    acc.copy_(torch.where(slot < lens, acc + w, torch.where((slot < lens + N) & (lens >= 0), w, acc)))
    return {"acc": st["acc"]}


def _commit(st):
    B, Hkv, N, S = st["B"], st["Hkv"], st["N"], st["S_max"]
    lens = st["lens"].long()
    i = torch.arange(N, device=lens.device)
    take = (i[None, :] < st["npath"][:, None]) & (lens >= 0)[:, None]
    dst = (lens.clamp(min=0)[:, None] + i).clamp(max=S - 1)
    src = torch.where(take, lens[:, None] + st["path"].long(), dst)        # [B][N]
    for name in ("k", "v", "acc", "pos"):
        t = st[name] if st[name].dim() == 4 else st[name][..., None]
        shape = (B, Hkv, N, t.shape[3])
        rows = torch.gather(t, 2, src[:, None, :, None].expand(shape))
        t.scatter_(2, dst[:, None, :, None].expand(shape), rows)
    st["lens_out"].copy_(torch.where(lens >= 0, lens + st["npath"], lens))
    return {n: st[n] for n in ("k", "v", "acc", "pos", "lens_out")}


def _evict(st):
    B, Hkv, S, keep, recent = st["B"], st["Hkv"], st["S_max"], st["keep"], st["recent"]
    lens = st["lens"].long()[:, None, None]
    slot = torch.arange(S, device=lens.device)[None, None]
    live = (slot < lens).expand(B, Hkv, S)
    pos = torch.where(live, st["pos"].long(), torch.full_like(st["pos"], -1).long())
    last = pos.amax(-1, keepdim=True)
    key = torch.where(live, torch.where(pos > last - recent, float("inf"), st["acc"]), float("-inf"))
    order = torch.argsort(key, dim=-1, descending=True, stable=True)
    kept = torch.zeros((B, Hkv, S), dtype=torch.bool, device=key.device)
    kept.scatter_(2, order[..., :keep], True)
    kept &= live
    # the r-th freed slot below `keep` takes the r-th kept slot at or past it
    mover = kept & (slot >= keep)
    rank = torch.where(mover, mover.long().cumsum(-1) - 1, torch.full_like(slot, keep))
    movers = torch.zeros((B, Hkv, keep + 1), dtype=torch.long, device=key.device)
    movers.scatter_(2, rank, slot.expand(B, Hkv, S))
    # (slots that do not move all land in the last, unused entry)
    low = slot[..., :keep]
    hole = ~kept[..., :keep] & (low < lens)
    src = torch.where(hole, torch.gather(movers, 2, (hole.long().cumsum(-1) - 1).clamp(min=0)), low.expand(B, Hkv, keep))
    new = lens.clamp(max=keep)
    src = torch.where(low < new, src, low)
    for name in ("k", "v"):
        rows = torch.gather(st[name], 2, src[..., None].expand(B, Hkv, keep, st["dh"]))
        st[name][:, :, :keep] = rows
    for name in ("acc", "pos"):
        out = st[name + "_out"][:, :, :keep]
        out.copy_(torch.where(low < new, torch.gather(st[name], 2, src), out))
    active = lens >= 0
    st["src"].copy_(torch.where(active, torch.where(low < new, src, -1), st["src"]))
    st["lens_out"].copy_(new[:, 0, 0])
    return {n: st[n] for n in ("k", "v", "acc_out", "pos_out", "src", "lens_out")}


# ------------------------------------------------------------------ the framework's operators

def _own(st):
    import flow_matching_action_loop_b200 as fr
    stream = torch.cuda.current_stream().cuda_stream
    op, B, Hkv, S, dh = st["op"], st["B"], st["Hkv"], st["S_max"], st["dh"]
    if op in ("attend", "weigh"):
        words = 0 if st["words"] is None else st["words"].data_ptr()
    if op == "attend":
        fr.fr_attention_tree(st["q"].data_ptr(), st["k"].data_ptr(), st["v"].data_ptr(), st["lens"].data_ptr(), words,
                             st["o"].data_ptr(), st["lse"].data_ptr(), B, st["Hq"], Hkv, st["N"], S, dh,
                             st["scratch"].data_ptr(), 40 << 20, stream)
        return {"o": st["o"], "lse": st["lse"]}
    if op == "weigh":
        fr.fr_attention_weights(st["q"].data_ptr(), st["k"].data_ptr(), st["lse"].data_ptr(), st["lens"].data_ptr(), words,
                                0 if st["use"] is None else st["use"].data_ptr(), st["acc"].data_ptr(), B, st["Hq"], Hkv,
                                st["N"], S, dh, stream)
        return {"acc": st["acc"]}
    dtype = fr.FR_DTYPE_F32 if st["dtype"] == "float32" else fr.FR_DTYPE_BF16
    if op == "commit":
        fr.fr_cache_commit(st["k"].data_ptr(), st["v"].data_ptr(), st["acc"].data_ptr(), st["pos"].data_ptr(),
                           st["lens"].data_ptr(), st["path"].data_ptr(), st["npath"].data_ptr(),
                           st["lens_out"].data_ptr(), B, Hkv, st["N"], S, dh, dtype, stream)
        return {n: st[n] for n in ("k", "v", "acc", "pos", "lens_out")}
    fr.fr_cache_evict(st["k"].data_ptr(), st["v"].data_ptr(), st["acc"].data_ptr(), st["pos"].data_ptr(),
                      st["lens"].data_ptr(), st["acc_out"].data_ptr(), st["pos_out"].data_ptr(),
                      st["lens_out"].data_ptr(), st["src"].data_ptr(), B, Hkv, S, dh, dtype, st["keep"], st["recent"],
                      stream)
    return {n: st[n] for n in ("k", "v", "acc_out", "pos_out", "src", "lens_out")}


def run(state):
    if own:
        return _own(state)
    return {"attend": _attend, "weigh": _weigh, "commit": _commit, "evict": _evict}[state["op"]](state)


def work(case):
    """Bytes and operations of one pass over the live part of the cache."""
    live = [n for n in _lens(case) if n >= 0]
    B, Hkv, dh = len(live), case["Hkv"], case["dh"]
    if case["op"] in ("attend", "weigh"):
        N, Hq = case["N"], case["Hq"]
        keys = sum(n + N for n in live)
        q = B * Hq * N * dh * 2
        if case["op"] == "attend":
            return {"bytes": keys * Hkv * dh * 2 * 2 + 2 * q + B * Hq * N * 4, "flops": 4.0 * keys * Hq * N * dh}
        return {"bytes": keys * Hkv * (dh * 2 + 8) + q + B * Hq * N * 4, "flops": 2.0 * keys * Hq * N * dh}
    row = dh * (4 if case["dtype"] == "float32" else 2)
    if case["op"] == "commit":
        # half of the drafted tokens on average, each read and written once
        return {"bytes": B * Hkv * case["N"] / 2 * 2 * (2 * row + 8), "flops": 0.0}
    keep, total = case["keep"], 0.0
    for n in live:
        kept = min(n, keep)
        # of the kept slots, those at or past `keep` move (on average their share of all slots); sums and
        # positions are read once each, those kept written once with their source
        moved = kept * max(0, n - keep) / max(1, n)
        total += moved * 2 * 2 * row + n * 8 + kept * 12
    return {"bytes": Hkv * total, "flops": 0.0}


# ------------------------------------------------------------------ the definition in 64 bits

def exact(case, seed):
    st = prepare(case, seed)
    op, Hkv = case["op"], case["Hkv"]
    lens = st["lens"].tolist()
    if op in ("attend", "weigh"):
        B, N, Hq, dh = case["B"], case["N"], case["Hq"], case["dh"]
        if 4.0 * Hq * N * dh * sum(max(n, 0) + N for n in lens) > 4e11:
            return None
        g = Hq // Hkv
        seen = np.tril(np.ones((N, N), bool))[None].repeat(B, 0)
        if st["words"] is not None:
            w = st["words"].cpu().numpy().view(np.uint32)
            seen = np.stack([(w[:, :, j // 32] >> np.uint32(j % 32)) & 1 for j in range(N)], axis=-1).astype(bool)
        counts = np.ones((B, N), bool)
        if st.get("use") is not None:
            u = st["use"].cpu().numpy().view(np.uint32)
            counts = np.stack([(u[:, j // 32] >> np.uint32(j % 32)) & 1 for j in range(N)], axis=-1).astype(bool)
        if op == "attend":
            o, lse = st["o"].double(), st["lse"].double()
        else:
            acc = st["acc"].double()
        for b in range(B):
            n = lens[b]
            if n < 0:
                continue
            # additive mask of the drafted block: 0 where token i sees token j
            block = torch.zeros(N, n + N, dtype=torch.float64, device="cuda")
            block[:, n:] = torch.from_numpy(np.where(seen[b], 0.0, -np.inf)).cuda()
            for h in range(Hq):
                keys = st["k"][b, h // g, :n + N].double()
                s = st["q"][b, h].double() @ keys.T / math.sqrt(dh) + block
                if op == "attend":
                    lse[b, h] = torch.logsumexp(s, -1)
                    o[b, :, h * dh:(h + 1) * dh] = torch.softmax(s, -1) @ st["v"][b, h // g, :n + N].double()
                else:
                    p = torch.exp(s - st["lse"][b, h].double()[:, None])
                    w = (p * torch.from_numpy(counts[b]).cuda().double()[:, None]).sum(0)
                    if h % g == 0:
                        acc[b, h // g, n:n + N] = 0
                    acc[b, h // g, :n + N] += w
        return {"o": o, "lse": lse} if op == "attend" else {"acc": acc}
    if op == "commit":
        path, npath = st["path"].tolist(), st["npath"].tolist()
        for b, n in enumerate(lens):
            if n < 0:
                continue
            picked = torch.tensor([n + j for j in path[b][:npath[b]]], dtype=torch.long, device="cuda")
            for name in ("k", "v", "acc", "pos"):
                st[name][b, :, n:n + npath[b]] = st[name][b][:, picked]
        st["lens_out"] = torch.tensor([n + c if n >= 0 else n for n, c in zip(lens, npath)], dtype=torch.int32)
        return {n: st[n] for n in ("k", "v", "acc", "pos", "lens_out")}
    keep, recent = case["keep"], case["recent"]
    for b, n in enumerate(lens):
        for h in range(Hkv if n >= 0 else 0):
            acc, pos = st["acc"][b, h, :n].cpu().numpy().astype(np.float64), st["pos"][b, h, :n].cpu().numpy()
            first = pos <= pos.max(initial=-1) - recent                    # unprotected slots sort after the others
            best = np.lexsort((np.arange(n), -acc * first, first))[:keep]
            low, high = np.setdiff1d(np.arange(min(n, keep)), best), np.sort(best[best >= keep])
            src = np.arange(min(n, keep))
            src[low] = high
            at = torch.from_numpy(src).cuda()
            for name in ("k", "v"):
                st[name][b, h, :len(src)] = st[name][b, h][at]
            for name in ("acc", "pos"):
                st[name + "_out"][b, h, :len(src)] = st[name][b, h][at]
            st["src"][b, h, :len(src)] = at.to(torch.int32)
            st["src"][b, h, len(src):] = -1
    st["lens_out"] = torch.tensor([min(n, keep) for n in lens], dtype=torch.int32)
    return {n: st[n] for n in ("k", "v", "acc_out", "pos_out", "src", "lens_out")}

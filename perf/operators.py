"""Cases of the operators that train and serve a calibrated attention layer.

Four operators, all over the library's skip lists or its blocks of tokens:

  bwd        gradients of block-sparse attention (q, k, v, the saved output and row log-sum-exps,
             and the output's gradient -> dq, dk, dv), with or without spatial-repetition heads
  transpose  the skip list by key block instead of by query block, which the gradients of the
             keys and values walk
  write      new keys and values quantised to 8 bits (e4m3) into a paged cache, one scale per
             block of tokens and head
  cached     attention over that cache, from a single query token per sequence upwards, over all
             of a sequence's blocks or those a skip list keeps

`own` chooses between the plain form of each (elementary torch operations in 32 bits, rounded
once at the end) and the library's entry points.
"""
import math

import torch

own = False

E4M3_MAX = 448.0
MIN_AMAX = 2.0 ** -100


# ----------------------------------------------------------------------------------
# cases
# ----------------------------------------------------------------------------------

def listed():
    return [
        # a unit-test-sized layer: what a gradient check or a toy model calls; latency counts
        dict(name="bwd_tiny", op="bwd", H=2, N=512, D=64, block=64, density=0.5, repeat=0),
        # a short clip of odd length, narrow heads, some query blocks with nothing kept
        dict(name="bwd_ragged", op="bwd", H=6, N=4999, D=64, block=128, density=0.4, repeat=0),
        # a shard of 4 heads of a 21-frame video layer (32760 tokens) at its calibrated density:
        # the training step's ordinary, and here largest, call
        dict(name="bwd_video", op="bwd", H=4, N=32760, D=128, block=128, density=0.35, repeat=0),
        # 5 latent frames of 45 x 80 with half of the heads computed on every fourth row only
        dict(name="bwd_repeat", op="bwd", H=4, N=18000, D=128, block=128, density=0.3, repeat=2,
             F=5, Hl=45, Wl=80, n_text=0, stride=4),
        # the list of one small layer, and of all 40 heads of a 75600-token layer
        dict(name="transpose_small", op="transpose", H=12, nq=64, nk=64, density=0.35),
        dict(name="transpose_large", op="transpose", H=40, nq=591, nk=591, density=0.25),
        # one new token for each of 32 running sequences
        dict(name="write_token", op="write", S=32, Hkv=8, M=1, D=128, block=128, longest=8192, ragged=True),
        # prompts of up to 4096 tokens going into the cache
        dict(name="write_prompt", op="write", S=8, Hkv=8, M=4096, D=128, block=128, longest=8192, ragged=True),
        # one stream, one query token, one latent frame cached (30 x 52 tokens): latency
        dict(name="cached_frame", op="cached", S=1, Hq=12, Hkv=12, M=1, D=128, block=128, longest=1560,
             ragged=False, density=1.0),
        # a batch of running sequences with shared key/value heads
        dict(name="cached_batch", op="cached", S=32, Hq=32, Hkv=8, M=1, D=128, block=128, longest=8192,
             ragged=True, density=1.0),
        # few streams over very long caches
        dict(name="cached_long", op="cached", S=4, Hq=32, Hkv=8, M=1, D=128, block=128, longest=131072,
             ragged=False, density=1.0),
        # several new tokens per sequence over the blocks that a mask keeps, narrow heads
        dict(name="cached_sparse", op="cached", S=8, Hq=16, Hkv=16, M=5, D=64, block=64, longest=32760,
             ragged=True, density=0.3),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["bwd", "bwd", "bwd", "transpose", "write", "cached", "cached", "cached"])
    if op == "bwd":
        D, block = rng.choice([64, 128]), rng.choice([64, 128])
        density = round(rng.uniform(0.05, 1.0), 3)
        if rng.random() < 0.3:
            F, Hl, Wl = rng.randint(1, 5), rng.randint(3, 45), rng.randint(3, 80)
            H, n_text, stride = rng.randint(1, 4), rng.choice([0, 0, 77, 256]), rng.randint(1, 5)
            return dict(op=op, H=H, N=F * Hl * Wl + n_text, D=D, block=block, density=min(density, 0.6),
                        repeat=rng.randint(1, H), F=F, Hl=Hl, Wl=Wl, n_text=n_text, stride=stride)
        N = _log(rng, 1, 16384)
        return dict(op=op, H=rng.randint(1, max(1, min(12, 32768 // N))), N=N, D=D, block=block,
                    density=density, repeat=0)
    if op == "transpose":
        n = _log(rng, 1, 591)
        return dict(op=op, H=rng.randint(1, 40), nq=n, nk=rng.choice([n, _log(rng, 1, 591)]),
                    density=round(rng.uniform(0.0, 1.0), 3))
    Hkv, D, block = rng.choice([1, 2, 4, 8, 12]), rng.choice([64, 128]), rng.choice([64, 128])
    longest = _log(rng, 1, 131072)
    S = rng.randint(1, max(1, min(64, 4 * 131072 * 8 // (longest * Hkv))))
    if op == "write":
        M = min(_log(rng, 1, 4096), longest)
        return dict(op=op, S=min(S, max(1, 32768 // M)), Hkv=Hkv, M=M, D=D, block=block, longest=longest,
                    ragged=rng.random() < 0.7)
    M = rng.choice([1, 1, 1, 2, 5, 16])
    return dict(op=op, S=S, Hq=Hkv * rng.choice([1, 2, 4, 5, 8]), Hkv=Hkv, M=M, D=D, block=block, longest=longest,
                ragged=rng.random() < 0.7, density=rng.choice([1.0, 1.0, round(rng.uniform(0.05, 0.9), 3)]))


# ----------------------------------------------------------------------------------
# inputs
# ----------------------------------------------------------------------------------

def _blocks(n, b):
    return (n + b - 1) // b


def _gen(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(1000003 * int(seed) + 17 * case["D" if "D" in case else "H"] + case.get("N", case.get("longest", 1)))
    return g


def _tokens(g, heads, n, D, smooth=None):
    """[heads, n, D]: noise plus smooth functions of the position.  Queries and keys share those
    (`smooth`), so that attention is stronger between near tokens."""
    noise = torch.randn(heads, n, D, device="cuda", generator=g)
    return noise if smooth is None else torch.baddbmm(noise, smooth[0].expand(heads, -1, -1), smooth[1])


def _smooth(g, heads, n, D):
    pos = torch.arange(n, device="cuda", dtype=torch.float32)
    freq = torch.rand(16, device="cuda", generator=g) * 0.05
    phi = torch.cos(pos[:, None] * freq + torch.arange(16, device="cuda"))
    return phi, torch.randn(heads, 16, D, device="cuda", generator=g) * 0.35


def _mask(g, rows, nq, nk, density):
    """uint8 [rows, nq, nk]: row i keeps round(density nk (1 + 0.3 cos(i))) blocks, the near ones more often
    than the far ones; below density 1 one row in 50 keeps nothing."""
    if density >= 1.0:
        return torch.ones(rows, nq, nk, dtype=torch.uint8, device="cuda")
    i = torch.arange(nq, device="cuda")[:, None]
    far = (i * (nk / nq) - torch.arange(nk, device="cuda")[None, :]).abs() / nk
    rank = (far + 0.5 * torch.rand(rows, nq, nk, device="cuda", generator=g)).argsort(-1).argsort(-1)
    count = (density * nk * (1 + 0.3 * torch.cos(i.double()))).round().clamp(1, nk)
    return ((rank < count) & (i % 50 != 7)).to(torch.uint8)


def _csr(mask):
    """Row pointers int32 and ascending kept columns int16 of a mask [rows, nq, nk], row-major."""
    ptr = torch.zeros(mask.shape[0] * mask.shape[1] + 1, dtype=torch.int32, device="cuda")
    ptr[1:] = mask.sum(-1, dtype=torch.int64).flatten().cumsum(0)
    return ptr, mask.nonzero()[:, 2].to(torch.int16)


def _anchors(c):
    """Token index of every anchor, and the anchor that each token takes (compacted order)."""
    F, Hl, Wl, s = c["F"], c["Hl"], c["Wl"], c["stride"]
    n = torch.arange(F * Hl * Wl, device="cuda")
    f, y, x = n // (Hl * Wl), n // Wl % Hl, n % Wl
    Ar = _blocks(Hl, s)
    of = (f * Ar + y // s) * Wl + x
    text = torch.arange(c["n_text"], device="cuda")
    return (torch.cat([n[y % s == 0], F * Hl * Wl + text]), torch.cat([of, F * Ar * Wl + text]))


def _forward(q, k, v, mask, block, scale):
    """The forward pass that a training step has behind it: fp32 output and row log-sum-exps."""
    s = torch.bmm(q, k.transpose(1, 2)).mul_(scale)
    keep = mask.bool().repeat_interleave(block, 1)[:, :q.shape[1]].repeat_interleave(block, 2)[:, :, :k.shape[1]]
    s.masked_fill_(~keep, -math.inf)
    lse = torch.logsumexp(s, 2)
    p = s.sub_(lse.masked_fill(lse == -math.inf, 0.0)[..., None]).exp_()
    return torch.bmm(p, v), lse


def prepare(case, seed):
    c, g = case, _gen(case, seed)
    if c["op"] == "bwd":
        H, N, D, B = c["H"], c["N"], c["D"], c["block"]
        smooth = _smooth(g, H, N, D)
        q, k, v = (_tokens(g, H, N, D, x).to(torch.bfloat16) for x in (smooth, smooth, None))
        do = (_tokens(g, H, N, D) * 0.05).to(torch.bfloat16)
        nb, R, scale = _blocks(N, B), c["repeat"], D ** -0.5
        mask = _mask(g, H, nb, nb, c["density"])
        o = torch.empty(H, N, D, dtype=torch.bfloat16, device="cuda")
        lse = torch.empty(H, N, dtype=torch.float32, device="cuda")
        if H > R:
            x, y = _forward(q[R:].float(), k[R:].float(), v[R:].float(), mask[R:], B, scale)
            o[R:], lse[R:] = x.to(o.dtype), y
        if R:
            at, of = _anchors(c)
            mask[:R, _blocks(at.numel(), B):] = 0
            x, y = _forward(q[:R, at].float(), k[:R].float(), v[:R].float(), mask[:R, :_blocks(at.numel(), B)], B, scale)
            o[:R], lse[:R] = x[:, of].to(o.dtype), y[:, of]
        t_mask = mask.transpose(1, 2).contiguous()
        return dict(c=c, q=q, k=k, v=v, o=o, do=do, lse=lse, mask=mask, list=_lists(mask), list_t=_lists(t_mask),
                    head_repeat=[h < R for h in range(H)])
    if c["op"] == "transpose":
        ptr, col = _csr(_mask(g, c["H"], c["nq"], c["nk"], c["density"]))
        return dict(c=c, ptr=ptr, col=col)

    # a paged cache: pages handed out in a random order, as a server that has run for a while has them
    S, Hkv, D, B, top = c["S"], c["Hkv"], c["D"], c["block"], c["longest"]
    M = c["M"]
    nb = _blocks(top, B)
    table = torch.randperm(S * nb, device="cuda", generator=g).to(torch.int32).view(S, nb)
    lengths = torch.full((S,), top, dtype=torch.int32, device="cuda")
    new = torch.full((S,), M, dtype=torch.int32, device="cuda")
    if c["ragged"]:
        lengths = (lengths * (0.25 + 0.75 * torch.rand(S, device="cuda", generator=g))).to(torch.int32).clamp_(min=1)
        new = (new * torch.rand(S, device="cuda", generator=g)).to(torch.int32).add_(1).clamp_(max=M)
        if S > 2:
            lengths[1] = 0                                              # a slot of the batch with no sequence
    new = torch.minimum(new, lengths)
    pages = S * nb
    if c["op"] == "write":
        kx, vx = (_tokens(g, S * Hkv, M, D).view(S, Hkv, M, D).to(torch.bfloat16) for _ in range(2))
        k8, v8 = (torch.randn(pages, Hkv, B, D, device="cuda", generator=g).mul_(90.0)
                  .clamp_(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn) for _ in range(2))
        ks, vs = (0.004 + 0.008 * torch.rand(pages, Hkv, device="cuda", generator=g) for _ in range(2))
        return dict(c=c, k8=k8, v8=v8, ks=ks, vs=vs, kx=kx, vx=vx, table=table, lengths=lengths, new=new)
    q = _tokens(g, S * c["Hq"], M, D).view(S, c["Hq"], M, D).to(torch.bfloat16)
    # keys and values drawn page by page: values in 8 bits that fill the type's range, and their scales
    k8, v8 = (torch.randn(pages, Hkv, B, D, device="cuda", generator=g, dtype=torch.bfloat16).mul_(100.0)
              .clamp_(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn) for _ in range(2))
    ks, vs = (0.006 + 0.008 * torch.rand(pages, Hkv, device="cuda", generator=g) for _ in range(2))
    s = dict(c=c, q=q, k8=k8, v8=v8, ks=ks, vs=vs, table=table, lengths=lengths, new=new, mask=None)
    if c["density"] < 1.0:
        s["mask"] = _mask(g, Hkv, S, nb, c["density"])
        s["list"] = _lists(s["mask"], order=False)
    return s


def _lists(mask, order=True):
    """The plan a program keeps for a mask: row pointers, kept columns and (order) the rows h << 16 | i,
    heads in order and longest rows first."""
    ptr, col = _csr(mask)
    H, nq, _ = mask.shape
    work = None
    if order:
        n = mask.sum(-1, dtype=torch.int64)
        i = torch.argsort(n, dim=1, descending=True, stable=True)
        work = ((torch.arange(H, device="cuda")[:, None] << 16) | i).to(torch.int32).flatten()
    return dict(H=H, nq=nq, nk=mask.shape[2], row_ptr=ptr, col_idx=col, work=work)


# ----------------------------------------------------------------------------------
# the plain forms
# ----------------------------------------------------------------------------------

def _keep(mask, block, nq, nk):
    return mask.bool().repeat_interleave(block, 1)[:, :nq].repeat_interleave(block, 2)[:, :, :nk]


def _grads(q, k, v, do, delta, lse, mask, block, scale):
    """fp32 dq, dk, dv of attention over the kept blocks: P = exp(S - LSE), dS = P (dO V^T - delta)."""
    keep = _keep(mask, block, q.shape[1], k.shape[1])
    p = torch.bmm(q, k.transpose(1, 2)).mul_(scale).sub_(lse[..., None]).exp_().masked_fill_(~keep, 0.0)
    dv = torch.bmm(p.transpose(1, 2), do)
    ds = torch.bmm(do, v.transpose(1, 2)).sub_(delta[..., None]).mul_(p)
    return torch.bmm(ds, k).mul_(scale), torch.bmm(ds.transpose(1, 2), q).mul_(scale), dv


def _plain_bwd(s, real=torch.float32):
    c, B, R = s["c"], s["c"]["block"], s["c"]["repeat"]
    q, k, v, o, do = (s[x].to(real) for x in ("q", "k", "v", "o", "do"))
    lse, scale = s["lse"].to(real), c["D"] ** -0.5
    delta = (o * do).sum(-1)
    if R == 0:
        return _grads(q, k, v, do, delta, lse, s["mask"], B, scale)
    # heads [0, R) compute anchor tokens only: the gradients of the tokens that take an anchor's output
    # add up at the anchor, and no other query of those heads has one
    at, of = _anchors(c)
    n = at.numel()
    do_a = torch.zeros(R, n, c["D"], dtype=real, device="cuda").index_add_(1, of, do[:R])
    delta_a = torch.zeros(R, n, dtype=real, device="cuda").index_add_(1, of, delta[:R])
    a = _grads(q[:R, at], k[:R], v[:R], do_a, delta_a, lse[:R, at], s["mask"][:R, :_blocks(n, B)], B, scale)
    dq = torch.zeros_like(q)
    dq[:R, at] = a[0]
    if R == c["H"]:
        return dq, a[1], a[2]
    b = _grads(q[R:], k[R:], v[R:], do[R:], delta[R:], lse[R:], s["mask"][R:], B, scale)
    dq[R:] = b[0]
    return dq, torch.cat([a[1], b[1]]), torch.cat([a[2], b[2]])


def _plain_transpose(s):
    c, ptr, col = s["c"], s["ptr"], s["col"].long()
    H, nq, nk = c["H"], c["nq"], c["nk"]
    row = torch.repeat_interleave(torch.arange(H * nq, device="cuda"), (ptr[1:] - ptr[:-1]).long(), output_size=col.numel())
    t_row = row // nq * nk + col
    order = torch.argsort(t_row, stable=True)
    t_ptr = torch.zeros(H * nk + 1, dtype=torch.int32, device="cuda")
    t_ptr[1:] = torch.zeros(H * nk, dtype=torch.int64, device="cuda").index_add_(0, t_row, torch.ones_like(t_row)).cumsum(0)
    return t_ptr, (row % nq)[order].to(torch.int16)


def _plain_write(s):
    """New tokens m < new[s] go to positions lengths[s] - new[s] + m.  A block's scale is that of its
    largest value, and never smaller than that of the tokens it held; those are rounded again if it grows."""
    c, table, lengths, new = s["c"], s["table"].long(), s["lengths"].long(), s["new"].long()
    S, M, B, Hkv = c["S"], c["M"], c["block"], c["Hkv"]
    first = lengths - new
    T = (M - 1 + B - 1) // B + 1                                        # blocks that M tokens can touch
    blk = first[:, None] // B + torch.arange(T, device="cuda")          # [S, T]
    live = blk * B < lengths[:, None]
    page = table.gather(1, blk.clamp(max=table.shape[1] - 1))
    pos = blk[..., None] * B + torch.arange(B, device="cuda")           # [S, T, B]
    isnew = (pos >= first[:, None, None]) & (pos < lengths[:, None, None])
    isold = (pos < first[:, None, None])[:, :, None, :, None]
    m = (pos - first[:, None, None]).clamp(0, M - 1).view(S, 1, T * B, 1)
    isnew = isnew[:, :, None, :, None]
    hit = live.flatten().nonzero()[:, 0]                                # touched (sequence, block) pairs
    where = page.flatten()[hit]
    for x, data, scales in ((s["kx"], s["k8"], s["ks"]), (s["vx"], s["v8"], s["vs"])):
        t = x.float().gather(2, m.expand(S, Hkv, T * B, c["D"])).view(S, Hkv, T, B, c["D"]).transpose(1, 2)
        old = data.view(torch.uint8)[page].view(torch.float8_e4m3fn).float()
        amax = torch.where(isnew, t, 0.0).abs().amax((3, 4))
        fresh = amax.clamp(min=MIN_AMAX) / E4M3_MAX
        held = torch.where(isold.any(3)[..., 0], scales[page], 0.0)
        scale = torch.maximum(fresh, held)
        inv = (1.0 / scale)[..., None, None]
        again = torch.where((scale > held)[..., None, None], old * (held[..., None, None] * inv), old)
        y = torch.where(isnew, t * inv, torch.where(isold, again, old)).clamp(-E4M3_MAX, E4M3_MAX)
        data.view(torch.uint8)[where] = y.flatten(0, 1)[hit].to(torch.float8_e4m3fn).view(torch.uint8)
        scales[where] = scale.flatten(0, 1)[hit]
    return s["k8"], s["v8"], s["ks"], s["vs"]


def _plain_cached(s, real=torch.float32):
    c, table = s["c"], s["table"].long()
    S, Hq, Hkv, M, D, B = c["S"], c["Hq"], c["Hkv"], c["M"], c["D"], c["block"]
    G, nb = Hq // Hkv, table.shape[1]

    def rows(data, scales):                                             # [S, Hkv, nb * B, D]
        x = data.view(torch.uint8)[table].view(torch.float8_e4m3fn).to(real).mul_(scales[table].to(real)[..., None, None])
        return x.transpose(1, 2).reshape(S, Hkv, nb * B, D)

    pos = torch.arange(nb * B, device="cuda")
    m = torch.arange(M, device="cuda")
    limit = torch.where(m < s["new"][:, None], (s["lengths"] - s["new"])[:, None] + m + 1, 0)      # [S, M]
    keep = (pos < limit[..., None])[:, None, None]                                          # [S, 1, 1, M, keys]
    if s["mask"] is not None:
        keep = keep & s["mask"].bool().transpose(0, 1).repeat_interleave(B, 2)[:, :, None, None]
    q = s["q"].to(real).view(S, Hkv, G * M, D)
    x = torch.matmul(q, rows(s["k8"], s["ks"]).transpose(2, 3)).mul_(D ** -0.5).view(S, Hkv, G, M, nb * B)
    x = x.masked_fill_(~keep, -math.inf)
    top = x.amax(-1, keepdim=True)
    top = top.masked_fill(top == -math.inf, 0.0)
    x = x.sub_(top).exp_()
    total = x.sum(-1, keepdim=True)
    values = rows(s["v8"], s["vs"])                     # keys that no sequence has yet hold anything
    values = values.masked_fill_((pos >= s["lengths"][:, None])[:, None, :, None], 0.0)
    o = torch.matmul(x.view(S, Hkv, G * M, nb * B), values).view(S, Hkv, G, M, D)
    o = (o / total.clamp(min=1e-30)).view(S, Hq, M, D)
    return o, (total.log() + top).view(S, Hq, M)


# ----------------------------------------------------------------------------------
# one pass
# ----------------------------------------------------------------------------------

def run(s):
    if own:
        return _own(s)
    c = s["c"]
    if c["op"] == "bwd":
        return tuple(x.to(torch.bfloat16) for x in _plain_bwd(s))
    if c["op"] == "transpose":
        return _plain_transpose(s)
    if c["op"] == "write":
        return _plain_write(s)
    o, lse = _plain_cached(s)
    return o.to(torch.bfloat16), lse


def _own(s):
    from calibrated_block_sparse_calib_b200 import ops
    c = s["c"]
    if c["op"] == "bwd":
        rows, cols = (ops.BlockList(block=c["block"], **s[x]) for x in ("list", "list_t"))
        if c["repeat"]:
            return ops.sparse_attn_bwd_repeat(s["q"], s["k"], s["v"], s["o"], s["do"], s["lse"], rows, s["head_repeat"],
                                              c["F"], c["Hl"], c["Wl"], c["n_text"], c["stride"], blist_t=cols)
        return ops.sparse_attn_bwd(s["q"], s["k"], s["v"], s["o"], s["do"], s["lse"], rows, blist_t=cols)
    if c["op"] == "transpose":
        return ops.transpose_csr(s["ptr"], s["col"], c["H"], c["nq"], c["nk"])
    cache = ops.KVCache(s["k8"], s["v8"], s["ks"], s["vs"])
    if c["op"] == "write":
        ops.cache_write(cache, s["kx"], s["vx"], s["table"], s["lengths"], new_lens=s["new"])
        return cache.k, cache.v, cache.k_scale, cache.v_scale
    keep = ops.BlockList(block=c["block"], **s["list"]) if s["mask"] is not None else None
    return ops.sparse_attn_cached(s["q"], cache, s["table"], s["lengths"], blist=keep, new_lens=s["new"], causal=True,
                                  return_lse=True)


# ----------------------------------------------------------------------------------
# what a pass cannot do without
# ----------------------------------------------------------------------------------

def _kept(c, nk):
    return 1.0 if c["density"] >= 1 else 0.98 * max(c["density"], 1 / nk)


def work(case):
    c = case
    if c["op"] == "bwd":
        # five products per kept pair of tokens; q, k, v, o, do in and dq, dk, dv out once, and the row statistics
        H, N, D = c["H"], c["N"], c["D"]
        rows = (H - c["repeat"]) * N
        if c["repeat"]:
            rows += c["repeat"] * (c["F"] * _blocks(c["Hl"], c["stride"]) * c["Wl"] + c["n_text"])
        return dict(bytes=8 * 2.0 * H * N * D + 4 * H * N, flops=10.0 * D * rows * N * _kept(c, _blocks(N, c["block"])))
    if c["op"] == "transpose":
        nnz = c["H"] * c["nq"] * c["nk"] * _kept(c, c["nk"])
        return dict(bytes=4.0 * nnz + 4.0 * c["H"] * (c["nq"] + c["nk"]), flops=0)
    share = 0.625 if c["ragged"] else 1.0
    if c["op"] == "write":
        n = c["S"] * c["Hkv"] * max(1.0, c["M"] * (0.5 if c["ragged"] and c["M"] > 1 else 1.0))
        return dict(bytes=2 * 3.0 * n * c["D"], flops=0)
    keys = c["S"] * c["Hkv"] * c["longest"] * share * _kept(c, _blocks(c["longest"], c["block"]))
    return dict(bytes=2.0 * keys * c["D"] + 4.0 * c["S"] * c["Hq"] * c["M"] * c["D"],
                flops=4.0 * keys * c["D"] * c["Hq"] // c["Hkv"] * c["M"])


# ----------------------------------------------------------------------------------
# the definitions in 64 bits
# ----------------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "bwd":
        return _exact_bwd(s)
    if case["op"] == "cached":
        return _exact_cached(s)
    if case["op"] == "write":
        return _exact_write(s)
    return None                                                         # whole numbers


def _exact_bwd(s):
    """Head by head and row block by row block: the gradients of sum(O * dO), with O's softmax written out
    and the saved statistics as they were given."""
    c = s["c"]
    H, N, D, B, scale = c["H"], c["N"], c["D"], c["block"], c["D"] ** -0.5
    dq, dk, dv = (torch.zeros(H, N, D, dtype=torch.float64, device="cuda") for _ in range(3))
    if c["repeat"]:
        at, of = _anchors(c)
    step = B * max(1, 4096 // B)
    col_block = torch.arange(N, device="cuda") // B
    for h in range(H):
        q, k, v, do, o = (s[x][h].double() for x in ("q", "k", "v", "do", "o"))
        lse, delta = s["lse"][h].double(), torch.einsum("nd,nd->n", do, o)
        rows = torch.arange(N, device="cuda")
        if s["head_repeat"][h]:
            rows = at
            do = torch.zeros(at.numel(), D, dtype=torch.float64, device="cuda").index_add_(0, of, do)
            delta = torch.zeros(at.numel(), dtype=torch.float64, device="cuda").index_add_(0, of, delta)
        for i in range(0, rows.numel(), step):
            r = rows[i:i + step]
            row_block = torch.arange(i, i + r.numel(), device="cuda") // B
            kept = s["mask"][h][row_block][:, col_block] != 0
            p = torch.where(kept, torch.exp(scale * q[r] @ k.T - lse[r, None]), 0.0)
            g = p * (do[i:i + step] @ v.T - delta[i:i + step, None])
            dq[h, r] = scale * g @ k
            dk[h] += scale * g.T @ q[r]
            dv[h] += p.T @ do[i:i + step]
    return dq, dk, dv


def _exact_cached(s):
    """Sequence by sequence over its own keys."""
    c = s["c"]
    G, M, D, B = c["Hq"] // c["Hkv"], c["M"], c["D"], c["block"]
    o = torch.zeros(c["S"], c["Hq"], M, D, dtype=torch.float64, device="cuda")
    lse = torch.full((c["S"], c["Hq"], M), -math.inf, dtype=torch.float64, device="cuda")
    lengths, new = s["lengths"].tolist(), s["new"].tolist()
    for i in range(c["S"]):
        L, n = lengths[i], new[i]
        if L == 0:
            continue
        page = s["table"][i, :_blocks(L, B)].long()
        k, v = ((x.view(torch.uint8)[page].view(torch.float8_e4m3fn).double() * y[page].double()[:, :, None, None]).transpose(0, 1).flatten(1, 2)[:, :L]
                for x, y in ((s["k8"], s["ks"]), (s["v8"], s["vs"])))
        a = torch.einsum("hgmd,hnd->hgmn", s["q"][i].double().view(c["Hkv"], G, M, D), k) / math.sqrt(D)
        at = torch.arange(L, device="cuda")
        ok = (at <= (L - n + torch.arange(M, device="cuda"))[:, None]) & (torch.arange(M, device="cuda") < n)[:, None]
        ok = ok[None, None].expand(c["Hkv"], G, M, L)
        if s["mask"] is not None:
            ok = ok & (s["mask"][:, i][:, at // B] != 0)[:, None, None]
        a = torch.where(ok, a, -math.inf)
        z = torch.logsumexp(a, -1)
        w = torch.where(ok, torch.exp(a - z.masked_fill(z == -math.inf, 0.0)[..., None]), 0.0)
        o[i] = torch.einsum("hgmn,hnd->hgmd", w, v).reshape(c["Hq"], M, D)
        lse[i] = z.reshape(c["Hq"], M)
    return o, lse


def _exact_write(s):
    """The scales, block by block that is written to; the values' rounding to 8 bits is part of what they are."""
    B = s["c"]["block"]
    ks, vs = s["ks"].double(), s["vs"].double()
    lengths, new, table = s["lengths"].tolist(), s["new"].tolist(), s["table"].tolist()
    for i, (L, n) in enumerate(zip(lengths, new)):
        for b in range((L - n) // B if n else 0, _blocks(L, B) if n else 0):
            lo, hi = max(L - n, b * B), min(L, (b + 1) * B)
            for x, scale in ((s["kx"], ks), (s["vx"], vs)):
                y = x[i, :, lo - (L - n):hi - (L - n)].double().abs().amax((1, 2)).clamp(min=MIN_AMAX) / E4M3_MAX
                scale[table[i][b]] = torch.maximum(y, scale[table[i][b]]) if lo > b * B else y
    return None, None, ks, vs

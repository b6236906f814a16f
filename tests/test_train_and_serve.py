"""The gradients, the transposed list and the 8-bit cache together, as a program would use them: calibrate a
slice, train through its list, write the trained keys and values into a cache and attend to them token by token
under the same mask.  Tolerances as in test_attn_bwd.py and test_kv_cache.py, whose checks are used."""
import math
import subprocess
import sys

import numpy as np
import pytest
import torch

import oracle
import test_attn_bwd
import test_kv_cache
from calibrated_block_sparse_calib_b200 import ops
from calibrated_block_sparse_calib_b200.calibrate import calibrate_slice
from conftest import ROOT, to64

pytestmark = pytest.mark.gpu


def test_calibrate_train_and_serve(tiny_inputs):
    wl, qkv = tiny_inputs
    s = wl.shape
    inputs = [tuple(x.cuda() for x in t) for t in qkv]
    mask, _, _ = calibrate_slice([(q, k) for q, k, _ in inputs], s.F, s.Hl, s.Wl, s.n_text, s.block, wl.extra["tau"])
    rows = ops.BlockList.from_mask(mask, s.block).validate()
    cols = rows.transpose().validate()
    q, k, v = inputs[0]
    H, N, D = q.shape
    target = inputs[1][2]

    # two steps on the values: O moves towards `target`, through autograd
    vw = v.clone().requires_grad_()
    kw = k.clone().requires_grad_()
    for _ in range(2):
        o = ops.sparse_attention(q, kw, vw, rows, cols)
        do = ((o.detach().float() - target.float()) * (2.0 / o.numel())).to(torch.bfloat16)
        gk, gv = torch.autograd.grad(o, (kw, vw), do)
        lse = ops.sparse_attn_fwd(q, kw.detach(), vw.detach(), rows, return_lse=True)[1]
        dq, dk, dv = ops.sparse_attn_bwd(q, kw.detach(), vw.detach(), o.detach(), do, lse, rows, cols)
        assert torch.equal(gk, dk) and torch.equal(gv, dv)
        test_attn_bwd._compare(q, kw.detach(), vw.detach(), o.detach(), do, lse, mask.cpu().numpy(), s.block, (dq, dk, dv))
        with torch.no_grad():
            vw -= (gv.float() * (0.1 * N)).to(torch.bfloat16)
            kw -= (gk.float() * (0.1 * N)).to(torch.bfloat16)

    # serve: two copies of the sequence, one cut short, in pages of the list's blocks
    k1, v1 = kw.detach(), vw.detach()
    nb = ops.nblocks(N, s.block)
    cache = ops.KVCache.allocate(2 * nb, H, s.block, D)
    table = torch.randperm(2 * nb, generator=torch.Generator().manual_seed(3)).to(torch.int32).view(2, nb).cuda()
    short = N - 100
    lengths = torch.tensor([N - 1, short - 1], dtype=torch.int32, device="cuda")
    both = lambda x: x[None].repeat(2, 1, 1, 1).contiguous()
    pad = lambda x: both(x)[:, :, :N - 1].contiguous()
    ops.cache_write(cache, pad(k1), pad(v1), table, lengths, new_lens=lengths)      # the prompts
    # the next token of each, and attention from it over the blocks that its query block keeps
    at = [N - 1, short - 1]
    new = [torch.stack([x[:, a:a + 1] for a in at]).contiguous() for x in (q, k1, v1)]
    lengths += 1
    ops.cache_write(cache, new[1], new[2], table, lengths)
    kept = torch.stack([mask[:, a // s.block] for a in at], 1).contiguous()          # [H, 2, nb]
    got, lse = ops.sparse_attn_cached(new[0], cache, table, lengths, blist=ops.BlockList.from_mask(kept, s.block), return_lse=True)
    ops.device_check()
    test_kv_cache._check(got, lse, new[0], cache, table, lengths.tolist(), [1, 1], D ** -0.5, True, kept.cpu().numpy())

    # and the cache stands for the trained keys and values: every value within half a step (2^-4 of it, 2^-10 of the scale
    # in the subnormal range), once more for blocks whose scale the last token raised
    for data, scale, x in ((cache.k, cache.k_scale, k1), (cache.v, cache.v_scale, v1)):
        y = (data.float() * scale[:, :, None, None])[table[0].long()].transpose(0, 1).reshape(H, -1, D)[:, :N]
        sc = scale[table[0].long()].t().repeat_interleave(s.block, 1)[:, :N, None]
        step = torch.maximum(x.float().abs() * 2.0 ** -4, sc * 2.0 ** -10) * 1.001
        assert bool(((y - x.float()).abs() <= 2 * step + step * 2.0 ** -4).all())
    # the full sequence's token attends as the forward pass does, up to the cache's rounding: against the same
    # attention of the rounded values, in 64 bits
    kd, vd = ((d.float() * sc[:, :, None, None])[table[0].long()].transpose(0, 1).reshape(H, -1, D)[:, :N]
              for d, sc in ((cache.k, cache.k_scale), (cache.v, cache.v_scale)))
    ref, _ = oracle.sparse_attention(to64(q), to64(kd), to64(vd), 1.0 / math.sqrt(D), s.block, mask.cpu().numpy(),
                                     q_blocks=[(N - 1) // s.block])
    # fp16 weights and bf16 output: 2^-11 sum P|v| and 2^-8 |O|, with sums of fewer than 2^10 terms (2^-14)
    most = np.abs(to64(vd)).max()
    err = np.abs(to64(got)[0, :, 0] - ref[:, N - 1])
    assert np.all(err <= (2.0 ** -10 + 2.0 ** -14) * most + 2.0 ** -8 * np.abs(ref[:, N - 1]))


def test_two_calls_at_once():
    """A backward pass and a cached attention on two streams at the same time give the bits they give alone."""
    H, N, D, B = 4, 3000, 128, 128
    q, k, v, do = test_attn_bwd._inputs(H, N, D, 21)
    nb = ops.nblocks(N, B)
    bl = ops.BlockList.from_mask(torch.ones(H, nb, nb, dtype=torch.uint8, device="cuda"), B)
    bt = bl.transpose()
    o, lse = ops.sparse_attn_fwd(q, k, v, bl, return_lse=True)
    cache, table = test_kv_cache._cache(np.random.default_rng(5), 3, 2, D, B, 40)
    lengths = torch.tensor([5000, 17, 3000], dtype=torch.int32, device="cuda")
    qs = torch.randn(3, 8, 1, D, device="cuda").to(torch.bfloat16)
    alone = (*ops.sparse_attn_bwd(q, k, v, o, do, lse, bl, bt), *ops.sparse_attn_cached(qs, cache, table, lengths, return_lse=True))
    streams = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    for _ in range(3):
        outs = []
        for st, call in zip(streams, (lambda: ops.sparse_attn_bwd(q, k, v, o, do, lse, bl, bt),
                                      lambda: ops.sparse_attn_cached(qs, cache, table, lengths, return_lse=True),
                                      lambda: ops.sparse_attn_bwd(q, k, v, o, do, lse, bl))):
            with torch.cuda.stream(st):
                outs.append(call())
        torch.cuda.synchronize()
        got = (*outs[0], *outs[1])
        assert all(torch.equal(a, b) for a, b in zip(alone, got))
        assert all(torch.equal(a, b) for a, b in zip(alone, outs[2]))
    ops.device_check()


@pytest.mark.parametrize("which", ["forward", "backward", "cached", "energy"])
def test_the_first_cuda_call_of_a_thread(which):
    """Each call as the first that a new thread makes: it has no CUDA context yet."""
    import threading
    H, N, D, B = 1, 200, 64, 64
    q, k, v, do = test_attn_bwd._inputs(H, N, D, 22)
    nb = ops.nblocks(N, B)
    bl = ops.BlockList.from_mask(torch.ones(H, nb, nb, dtype=torch.uint8, device="cuda"), B)
    bt = bl.transpose()
    o, lse = ops.sparse_attn_fwd(q, k, v, bl, return_lse=True)
    cache, table = test_kv_cache._cache(np.random.default_rng(5), 1, 1, D, B, 4)
    lengths = torch.tensor([200], dtype=torch.int32, device="cuda")
    grads = [torch.empty_like(q) for _ in range(3)]
    out, energy = torch.empty(1, 1, 1, D, dtype=torch.bfloat16, device="cuda"), torch.empty(H, nb, nb, device="cuda")
    calls = {"forward": lambda: ops.sparse_attn_fwd(q, k, v, bl, out=o, lse=lse),
             "backward": lambda: ops.sparse_attn_bwd(q, k, v, o, do, lse, bl, bt, dq=grads[0], dk=grads[1], dv=grads[2]),
             "cached": lambda: ops.sparse_attn_cached(q[:, None, :1].contiguous(), cache, table, lengths, out=out),
             "energy": lambda: ops.block_energy(q, k, B, out=energy)}
    raised = []

    def body():
        try:
            calls[which]()
        except Exception as e:                                     # noqa: BLE001
            raised.append(e)

    torch.cuda.synchronize()
    t = threading.Thread(target=body)
    t.start()
    t.join()
    assert not raised, raised
    ops.device_check()


def test_the_first_cuda_call_of_a_process():
    """A call that takes no tensor, before anything else has touched CUDA."""
    body = "from calibrated_block_sparse_calib_b200 import ops; ops.device_check(); print('ok')"
    res = subprocess.run([sys.executable, "-c", body], capture_output=True, text=True, timeout=240, cwd=ROOT)
    assert res.returncode == 0 and res.stdout.strip() == "ok", res.stderr[-2000:]

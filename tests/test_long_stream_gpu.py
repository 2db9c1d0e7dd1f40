"""The long-stream operators together, as a server and a trainer use them."""
import numpy as np
import pytest
import torch

import block_sparse_attention_38_b200 as bsa
from oracle import long_stream as o

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bits", [4, 16])
def test_prompt_then_tokens(bits):
    """A padded batch of prompts is prefilled with a window and sinks, its keys and
    values go into the cache, and three tokens of each sequence are decoded; every
    step against the oracle on the values that the cache stands for.

    Tolerances: those of the forward (2^-8 |O| + 2^-8 max|v|) and of a decode step
    (2^-8 |O| + 2^-10 max|v|), |v| below 5."""
    B, H, Hkv, N, L, d, W, S = 3, 8, 2, 300, 310, 128, 90, 4
    g = torch.Generator().manual_seed(31)
    lens = [300, 157, 3]

    def rand(*shape):
        return torch.randn(shape, generator=g).to(torch.bfloat16)

    q, k, v = rand(B, H, N, d), rand(B, Hkv, N, d), rand(B, Hkv, N, d)
    n = torch.tensor(lens, dtype=torch.int32, device="cuda")
    out, _ = bsa.window_forward(q.cuda(), k.cuda(), v.cuda(), W, S, lens=n)
    want, _ = o.window_forward(q, k, v, W, S, d ** -0.5, lens)
    np.testing.assert_allclose(out.float().cpu().numpy(), want, rtol=2.0 ** -8, atol=2.0 ** -8 * 5)

    zero = torch.zeros(B, dtype=torch.int32, device="cuda")
    if bits == 4:
        cache = bsa.q4_cache(B, Hkv, L, d)
        bsa.q4_write(cache, k.cuda(), v.cuda(), zero, lens=n)
        kept = [o.values(*o.quantise(x)) for x in (k, v)]
    else:
        kc, vc = (torch.zeros(B, Hkv, L, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        kc[:, :, :N], vc[:, :, :N] = k.cuda(), v.cuda()
        kept = [x.double().numpy() for x in (k, v)]
    kept = [np.concatenate([x, np.zeros((B, Hkv, L - N, d))], 2) for x in kept]
    for _ in range(3):
        n += 1
        lens = [x + 1 for x in lens]
        q1, k1, v1 = rand(B, H, d), rand(B, Hkv, d), rand(B, Hkv, d)
        for x, new in zip(kept, (k1, v1)):
            new = o.values(*o.quantise(new)) if bits == 4 else new.double().numpy()
            for b in range(B):
                x[b, :, lens[b] - 1] = new[b]
        if bits == 4:
            out, lse = bsa.q4_window_decode(q1.cuda(), cache, n, W, S, k_new=k1.cuda(), v_new=v1.cuda())
        else:
            out, lse = bsa.window_decode(q1.cuda(), kc, vc, n, W, S, k_new=k1.cuda(), v_new=v1.cuda())
        want, lw = o.decode(q1, *kept, lens, lambda b, h, t: o.window_rows(t, W, S), d ** -0.5)
        np.testing.assert_allclose(out.float().cpu().numpy(), want, rtol=2.0 ** -8 + 2.0 ** -20, atol=2.0 ** -10 * 5)
        np.testing.assert_allclose(lse.cpu().numpy(), lw, atol=2.0 ** -13)
    if bits == 4:  # what a later prefill chunk would read back
        kr, _ = bsa.q4_read(cache, zero, L, lens=n)
        for b in range(B):
            np.testing.assert_allclose(kr[b, :, :lens[b]].float().cpu().numpy(), kept[0][b, :, :lens[b]],
                                       rtol=2.0 ** -8 + 2.0 ** -20)
            assert float(kr[b, :, lens[b]:].abs().sum()) == 0
    assert bsa.stream_status() == 0


def test_block_pattern_over_both_caches_agrees():
    """bsa_decode over bf16 and q4_decode over the same rows in 4 bits, with the
    values that the codes stand for (exact in bf16 here) in the bf16 cache."""
    B, H, L, d, bs = 2, 4, 512, 128, 64
    g = torch.Generator().manual_seed(32)
    # codes times 1/2 minus 4: scale and minimum exact, values exact in bf16
    k, v = (torch.randint(0, 16, (B, H, L, d), generator=g) / 2 - 4 for _ in range(2))
    k[..., 0::32], v[..., 0::32], k[..., 1::32], v[..., 1::32] = -4, -4, 3.5, 3.5
    k, v = k.to(torch.bfloat16), v.to(torch.bfloat16)
    rp, ci = bsa.build_pattern(bsa.LOGLINEAR, L // bs, H, log_kmax=2, anchors=(0,), causal=True)
    rp, ci = torch.from_numpy(rp).cuda(), torch.from_numpy(ci).cuda()
    n = torch.tensor([512, 301], dtype=torch.int32, device="cuda")
    cache = bsa.q4_cache(B, H, L, d)
    bsa.q4_write(cache, k.cuda(), v.cuda(), torch.zeros(B, dtype=torch.int32, device="cuda"))
    kr, vr = bsa.q4_read(cache, torch.zeros(B, dtype=torch.int32, device="cuda"), L)
    assert torch.equal(kr.cpu(), k) and torch.equal(vr.cpu(), v)
    q = torch.randn(B, H, d, generator=g).to(torch.bfloat16).cuda()
    a, la = bsa.decode(q, k.cuda(), v.cuda(), n, rp, ci, bs, d ** -0.5)
    b, lb = bsa.q4_decode(q, cache, n, rp, ci, bs)
    assert bsa.stream_status() == 0 and bsa.decode_status() == 0
    # two bf16 roundings (2^-8 each), and 2^-10 max|v| for the weights' rounding to fp16
    np.testing.assert_allclose(a.float().cpu(), b.float().cpu(), rtol=2.0 ** -7, atol=2.0 ** -10 * 4)
    np.testing.assert_allclose(la.cpu(), lb.cpu(), atol=2.0 ** -12)


def test_gradients_of_a_loss_along_a_direction():
    """loss = sum(w * O): its gradients by window_backward against differences of the
    oracle's loss along a random direction, in fp64.

    The directional derivative is a sum of 3 * B * N * d products of gradient and
    direction; each gradient element is off by less than 2^-7 of the gradient's root
    mean square r in the root mean square, so the sum by 2^-7 r sqrt(count), five times
    over for a bound."""
    B, H, Hkv, N, d, W, S = 1, 4, 2, 200, 64, 40, 3
    g = torch.Generator().manual_seed(33)
    q, k, v = (torch.randn(B, h, N, d, generator=g).to(torch.bfloat16) for h in (H, Hkv, Hkv))
    w = torch.randn(B, H, N, d, generator=g).to(torch.bfloat16)
    out, lse = bsa.window_forward(q.cuda(), k.cuda(), v.cuda(), W, S)
    grads = bsa.window_backward(q.cuda(), k.cuda(), v.cuda(), out, w.cuda(), lse, W, S)
    assert bsa.stream_status() == 0
    xs = [x.double().numpy() for x in (q, k, v)]
    steps = [np.random.default_rng(i).standard_normal(x.shape) for i, x in enumerate(xs)]
    eps = 1e-5
    hi, lo = ((o.window_forward(*[x + e * s for x, s in zip(xs, steps)], W, S, d ** -0.5)[0] * w.double().numpy()).sum()
              for e in (eps, -eps))
    slope = sum((gr.double().cpu().numpy() * s).sum() for gr, s in zip(grads, steps))
    size = sum((gr.double().cpu().numpy() ** 2).sum() for gr in grads) ** 0.5
    assert abs(slope - (hi - lo) / (2 * eps)) <= 5 * 2.0 ** -7 * size

"""attn_rope against the 64-bit oracle: pairings, axes, partial rotation, layouts,
far and negative positions, its gradient, in-place and captured calls."""
import numpy as np
import pytest
import torch

import attention_backward_bwd_gb300 as ab
from oracle import cache_oracle as co
from tests.cache_helpers import DT, HALF_STEP, SMALLEST, f64

pytestmark = pytest.mark.gpu


def _inv(n, base=10000.0):
    return (1.0 / base ** (torch.arange(n, dtype=torch.float64) / n)).float()


def _positions(axes, lead, hi, seed, lo=0):
    g = torch.Generator().manual_seed(seed)
    return torch.randint(lo, hi, (axes, *lead), generator=g, dtype=torch.int64).to(torch.int32)


def _check(got, x, pos, inv, sections, interleaved, inverse):
    """Sines and cosines to 2^-20 (angle 2^-22 of a radian, sincospi 2 steps), two
    products and a sum in fp32 (3 * 2^-24), one rounding to the type."""
    t = x.shape[:-2]
    flat = f64(x).reshape(-1, *x.shape[-2:])
    ref = co.rope(flat, pos.reshape(len(sections), -1).numpy(), inv.numpy(), sections, interleaved,
                  inverse).reshape(*t, *x.shape[-2:])
    n = len(inv)
    size = np.zeros_like(ref)
    a = np.abs(flat).reshape(ref.shape)
    i = np.arange(n)
    u, v = (2 * i, 2 * i + 1) if interleaved else (i, i + n)
    size[..., u] = size[..., v] = a[..., u] + a[..., v]
    bound = HALF_STEP[x.dtype] * np.abs(ref) + 2.0 ** -19 * size + SMALLEST[x.dtype]
    off = np.abs(f64(got) - ref) - bound
    assert (off <= 0).all(), f"{off.max():.3e} beyond the bound"
    assert np.array_equal(f64(got)[..., 2 * n:], f64(x)[..., 2 * n:])


CASES = [
    # dtype, lead, hq, hk, D, n_freq, sections, interleaved, far
    ("bf16", (1,), 1, 1, 8, 4, (4,), False, 10),
    ("fp16", (1, 1), 2, 1, 64, 32, (32,), True, 10),
    ("bf16", (2, 37), 8, 2, 128, 64, (16, 24, 24), False, 50000),
    ("fp16", (61,), 4, 4, 96, 32, (8, 24), True, 2000000),
    ("bf16", (1000,), 3, 1, 80, 20, (11, 9), True, 5000),     # 4-frequency chunks
    ("fp16", (3, 129), 2, 2, 72, 11, (5, 2, 2, 2), False, 700),  # pair by pair
    ("bf16", (77,), 2, 2, 256, 11, (0, 11), True, 700),
    ("bf16", (5000,), 20, 1, 256, 128, (128,), False, 2**31 - 1),
    ("fp16", (4100,), 2, 2, 40, 8, (3, 5), False, 100),
]


@pytest.mark.parametrize("case", CASES, ids=[f"{c[0]}-{c[1]}-d{c[4]}-f{c[5]}" for c in CASES])
@pytest.mark.parametrize("inverse", [False, True])
def test_rope_matches_the_oracle(case, inverse):
    dt, lead, hq, hk, d, n, sec, inter, far = case
    g = torch.Generator().manual_seed(3)
    q = torch.randn(*lead, hq, d, generator=g).to(DT[dt])
    k = torch.randn(*lead, hk, d, generator=g).to(DT[dt])
    pos, inv = _positions(len(sec), lead, far, 4), _inv(n)
    rq, rk = ab.attn_rope(q.cuda(), k.cuda(), pos.cuda(), inv.cuda(), sec, inter, inverse)
    _check(rq, q, pos, inv, sec, inter, inverse)
    _check(rk, k, pos, inv, sec, inter, inverse)


def test_negative_positions_and_one_axis_without_its_dimension():
    q = torch.randn(50, 2, 64).half()
    pos, inv = _positions(1, (50,), 2**31 - 1, 7, lo=-2**31), _inv(32, 100.0)
    rq, rk = ab.attn_rope(q.cuda(), None, pos[0].cuda(), inv.cuda())
    assert rk is None
    _check(rq, q, pos, inv, (32,), False, False)


def test_strided_views_of_a_joint_projection_rotate_in_place():
    b, s, hq, hk, d = 2, 70, 4, 2, 64
    joint = torch.randn(b, s, hq + 2 * hk, d).to(torch.bfloat16).cuda()
    before = joint.clone()
    q, k, v = joint.split([hq, hk, hk], dim=2)
    pos, inv = _positions(2, (b, s), 900, 8), _inv(16)
    rq, rk = ab.attn_rope(q, k, pos.cuda(), inv.cuda(), (7, 9), out_q=q, out_k=k)
    assert rq is q and rk is k
    _check(q, before[:, :, :hq].cpu(), pos, inv, (7, 9), False, False)
    _check(k, before[:, :, hq:hq + hk].cpu(), pos, inv, (7, 9), False, False)
    assert torch.equal(v, before[:, :, hq + hk:])
    # heads before positions in memory
    x = torch.randn(b, hq, s, d).half().cuda().transpose(1, 2)
    rx, _ = ab.attn_rope(x, None, pos.cuda(), inv.cuda(), (7, 9), interleaved=True)
    _check(rx, x.cpu(), pos, inv, (7, 9), True, False)


def test_inverse_is_the_gradient():
    """<rope(x + h e) - rope(x - h e), dy> / 2h in 64 bits against inverse=True of dy."""
    t, h, d, n = 3, 2, 16, 6
    g = torch.Generator().manual_seed(1)
    x, dy = (torch.randn(t, h, d, generator=g).half() for _ in range(2))
    pos, inv = _positions(2, (t,), 40, 2), _inv(n, 50.0)
    got = f64(ab.attn_rope(dy.cuda(), None, pos.cuda(), inv.cuda(), (4, 2), inverse=True)[0])
    step = 1e-5
    for i in np.ndindex(t, h, d):
        e = np.zeros((t, h, d))
        e[i] = step
        diff = (co.rope(f64(x) + e, pos.numpy(), inv.numpy(), (4, 2)) -
                co.rope(f64(x) - e, pos.numpy(), inv.numpy(), (4, 2))) / (2 * step)
        want = (diff * f64(dy)).sum()
        assert abs(got[i] - want) <= 2.0 ** -11 * abs(want) + 2.0 ** -18 + 1e-8


def test_training_step_with_rotary_positions():
    """rope, attn_fwd, attn_bwd, rope back: dq and dk against the whole chain in 64 bits
    (the tolerances of the backward's own tests)."""
    from oracle import attn_oracle
    from tests.gpu_helpers import assert_close
    b, s, hq, hk, d = 1, 130, 4, 2, 64
    g = torch.Generator().manual_seed(9)
    q, k, v, do = (torch.randn(b, s, h, d, generator=g).to(torch.bfloat16) for h in (hq, hk, hk, hq))
    pos, inv = _positions(3, (b, s), 500, 10), _inv(32)
    rot = (pos.cuda(), inv.cuda(), (8, 12, 12))
    rq, rk = ab.attn_rope(q.cuda(), k.cuda(), *rot)
    o, lse = ab.attn_fwd(rq, rk, v.cuda(), causal=True)
    dq, dk, dv = ab.attn_bwd(rq, rk, v.cuda(), o, lse, do.cuda(), causal=True)
    ab.attn_rope(dq, dk, *rot, inverse=True, out_q=dq, out_k=dk)
    ab.check_device_status()
    turn = lambda x, back: co.rope(x[0], pos[:, 0].numpy(), inv.numpy(), (8, 12, 12), False, back)[None]  # noqa: E731
    ref = attn_oracle.mha_backward(turn(f64(q), False), turn(f64(k), False), f64(v), f64(do), d ** -0.5, True)
    assert_close("dQ", dq, turn(ref["dQ"], True))
    assert_close("dK", dk, turn(ref["dK"], True))
    assert_close("dV", dv, ref["dV"])


def test_captured_call_on_another_stream_reads_new_values():
    q = torch.randn(40, 4, 64).half().cuda()
    pos, inv = _positions(1, (40,), 300, 5), _inv(32)
    dpos, dinv, out = pos.cuda(), inv.cuda(), torch.empty_like(q)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    ab.attn_rope(q, None, dpos, dinv, out_q=out, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        ab.attn_rope(q, None, dpos, dinv, out_q=out)
    new = torch.randn(40, 4, 64).half()
    q.copy_(new)
    dpos.copy_(pos + 17)
    g.replay()
    torch.cuda.synchronize()
    _check(out, new, pos + 17, inv, (32,), False, False)


def test_no_tokens():
    q = torch.empty(0, 2, 64, dtype=torch.float16, device="cuda")
    inv = _inv(32).cuda()
    rq, _ = ab.attn_rope(q, None, torch.empty(0, dtype=torch.int32, device="cuda"), inv)
    assert rq.shape == q.shape

"""pa_kv_append_rope on the GPU against the rotation in 64 bits (GPU)."""
import pytest
import torch

from paged_kv_varlen_flashattention_gb300 import binding
from tests import _q8

pytestmark = pytest.mark.gpu


def _tol(y, mag, dtype):
    """Half a step of the type at y (and of its subnormals), plus three fp32 roundings of the
    products' magnitudes."""
    t = _q8.TORCH[dtype]
    return torch.finfo(t).eps / 2 * y.abs() * (1 + 2 ** -10) + 3 * 2.0 ** -24 * mag + torch.finfo(t).smallest_normal * \
        torch.finfo(t).eps / 2


def run(sk, n, P=32, H=4, Hkv=2, D=64, rot=None, dtype="bf16", interleaved=False, seed=0, in_place=False, fused=False,
        behind=0, with_q=True):
    """One call; checks q, the new slots, and that every other slot kept its bits."""
    rot = D if rot is None else rot
    g = torch.Generator().manual_seed(seed)
    bt, nb = _q8.block_table(sk, P, seed + 1)
    t = _q8.TORCH[dtype]
    total = sum(n) + behind
    if fused:  # q, k and v as views of one projection's rows
        rows = torch.randn((total, (H + 2 * Hkv) * D), generator=g).to(t).cuda()
        q = rows[:, :H * D].view(total, H, D)
        kn = rows[:, H * D:(H + Hkv) * D].view(total, Hkv, D)
        vn = rows[:, (H + Hkv) * D:].view(total, Hkv, D)
    else:
        q, kn, vn = (torch.randn((total, h, D), generator=g).to(t).cuda() for h in (H, Hkv, Hkv))
    kc, vc = (torch.randn((nb, P, Hkv, D), generator=g).to(t) for _ in range(2))
    cos, sin = _q8.tables(max(sk) + 3, rot)
    kd, vd = kc.cuda(), vc.cuda()
    q0, kn0, vn0 = q.cpu(), kn.cpu(), vn.cpu()
    marker = torch.full_like(q, 7.0) if not in_place else q
    got = binding.kv_append_rope(kn, vn, _q8.cu(n).cuda(), _q8.cu(sk).cuda(), bt.cuda(), kd, vd, cos.cuda(), sin.cuda(),
                                 q=q if with_q else None, q_out=marker if with_q else None, interleaved=interleaved)
    assert binding.device_status() == 0, binding.last_error()
    pos, real = _q8.positions(n, sk), sum(n)
    if with_q:
        yq, mq = _q8.rotate(q0[:real], pos, cos, sin, interleaved)
        err = (got.cpu().double()[:real] - yq).abs()
        assert (err <= _tol(yq, mq, dtype)).all(), float(err.max())
        if behind:
            assert torch.equal(got.cpu()[real:], q0[real:] if in_place else torch.full_like(q0[real:], 7.0))
    else:
        assert got is None
    yk, mk = _q8.rotate(kn0[:real], pos, cos, sin, interleaved)
    seq = torch.repeat_interleave(torch.arange(len(n)), torch.tensor(n))
    blk, slot = bt[seq, pos // P].long(), pos % P
    err = (kd.cpu()[blk, slot].double() - yk).abs()
    assert (err <= _tol(yk, mk, dtype)).all(), float(err.max())
    vc[blk, slot] = vn0[:real]
    assert torch.equal(vd.cpu().view(torch.int16), vc.view(torch.int16))
    kc[blk, slot] = kd.cpu()[blk, slot]
    assert torch.equal(kd.cpu().view(torch.int16), kc.view(torch.int16))


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_rope_mixed_batch(dtype, interleaved):
    """Whole prompts, single tokens, chunks over page borders and sequences without new tokens."""
    run([70, 33, 1, 96, 40, 5, 300], [7, 0, 1, 96, 40, 2, 129], dtype=dtype, interleaved=interleaved)


@pytest.mark.parametrize("D,rot,H,Hkv,P", [(128, 128, 32, 8, 64), (80, 80, 6, 3, 96), (256, 64, 5, 1, 32),
                                           (512, 512, 2, 2, 256), (72, 32, 3, 1, 32), (16, 16, 1, 1, 32), (96, 48, 15, 3, 64)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_rope_head_shapes(D, rot, H, Hkv, P, interleaved):
    run([513, 1, 257, 90], [100, 1, 30, 90], P=P, H=H, Hkv=Hkv, D=D, rot=rot, interleaved=interleaved, seed=D)


def test_rope_one_token():
    run([1], [1])


def test_rope_views_of_one_projection_in_place():
    run([90, 17, 64], [30, 17, 1], D=128, fused=True, in_place=True)


def test_rope_without_q():
    run([90, 17, 64], [30, 17, 1], D=128, with_q=False)


@pytest.mark.parametrize("in_place", [False, True])
def test_rope_rows_behind_the_last_sequence_stay(in_place):
    run([40, 9], [8, 9], behind=13, in_place=in_place)


def test_rope_many_tokens_warp_per_token():
    run([3000, 50], [2990, 1], D=128, H=8, Hkv=2, seed=3)


def test_rope_no_tokens_and_no_sequences():
    run([5, 9], [0, 0])
    e = torch.empty((0, 2, 64), dtype=torch.bfloat16, device="cuda")
    kc = torch.ones((2, 32, 2, 64), dtype=torch.bfloat16, device="cuda")
    cos, sin = (x.cuda() for x in _q8.tables(4, 64))
    z = torch.zeros(1, dtype=torch.int32, device="cuda")
    binding.kv_append_rope(e, e, z, z, torch.zeros((0, 1), dtype=torch.int32, device="cuda"), kc, kc.clone(), cos, sin)
    assert binding.device_status() == 0 and (kc == 1).all()


def test_rope_position_past_the_tables_is_reported_others_written():
    n, sk, P = [2, 2], [40, 3], 32
    bt, nb = _q8.block_table(sk, P, 1)
    kc = torch.zeros((nb, P, 1, 64), dtype=torch.bfloat16, device="cuda")
    vc = torch.zeros_like(kc)
    one = torch.ones((4, 1, 64), dtype=torch.bfloat16, device="cuda")
    cos, sin = (x.cuda() for x in _q8.tables(39, 64))  # position 39, the second token's, is missing
    q = torch.full((4, 1, 64), 5.0, dtype=torch.bfloat16, device="cuda")
    got = binding.kv_append_rope(one, one, _q8.cu(n).cuda(), _q8.cu(sk).cuda(), bt.cuda(), kc, vc, cos, sin, q=q,
                                 q_out=torch.zeros_like(q))
    assert binding.STATUS[binding.device_status()] == "PA_ERR_DEVICE_BOUNDS"
    assert (vc.cpu()[int(bt[0, 1]), 38 - 32] == 1).all() and (vc.cpu()[int(bt[0, 1]), 39 - 32] == 0).all()
    assert (vc.cpu()[int(bt[1, 0]), 1:3] == 1).all()
    assert (got.cpu()[1] == 0).all() and (got.cpu()[0] != 0).any() and (got.cpu()[2] != 0).any()


def test_rope_bad_block_is_reported_and_its_q_is_rotated():
    n, sk, P = [3, 4], [3, 4], 32
    bt, nb = _q8.block_table(sk, P, 1)
    bt[0, 0] = nb + 2
    kc = torch.zeros((nb, P, 1, 64), dtype=torch.bfloat16, device="cuda")
    vc = torch.zeros_like(kc)
    one = torch.ones((7, 1, 64), dtype=torch.bfloat16, device="cuda")
    cos, sin = (x.cuda() for x in _q8.tables(8, 64))
    got = binding.kv_append_rope(one, one, _q8.cu(n).cuda(), _q8.cu(sk).cuda(), bt.cuda(), kc, vc, cos, sin, q=one,
                                 q_out=torch.zeros_like(one))
    assert binding.STATUS[binding.device_status()] == "PA_ERR_DEVICE_BOUNDS"
    assert (got.cpu()[0] == 1).all()  # position 0: not turned
    assert int((vc != 0).sum()) == 4 * 64


def test_rope_captured_and_replayed():
    """A captured call reads the lengths of the replay."""
    P, D = 32, 64
    bt = torch.arange(4, dtype=torch.int32)[None].cuda()
    kc = torch.zeros((4, P, 1, D), dtype=torch.bfloat16, device="cuda")
    vc = torch.zeros_like(kc)
    x = torch.randn((1, 1, D), device="cuda").bfloat16()
    cos, sin = (t.cuda() for t in _q8.tables(128, D))
    new, keys = _q8.cu([1]).cuda(), _q8.cu([1]).cuda()
    q = torch.empty_like(x)
    call = lambda: binding.kv_append_rope(x, x, new, keys, bt, kc, vc, cos, sin, q=x, q_out=q)  # noqa: E731
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        call()
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        call()
    for m in (1, 2, 33, 128):
        keys[1] = m
        graph.replay()
        torch.cuda.synchronize()
        y, mag = _q8.rotate(x.cpu(), torch.tensor([m - 1]), cos.cpu(), sin.cpu(), False)
        assert ((kc.cpu()[(m - 1) // P, (m - 1) % P].double() - y[0]).abs() <= _tol(y, mag, "bf16")[0]).all()
        assert torch.equal(vc[(m - 1) // P, (m - 1) % P], x[0])
    assert binding.device_status() == 0

"""pa_kv_append_q8 on the GPU against the 8-bit append in 64 bits (GPU)."""
import pytest
import torch

from paged_kv_varlen_flashattention_gb300 import binding
from tests import _q8

pytestmark = pytest.mark.gpu


class Step:
    """A pool and a batch; ``call`` appends on the GPU, ``check`` compares with 64 bits."""

    def __init__(self, sk, n, P=32, H=4, Hkv=2, D=64, rot=None, dtype="bf16", interleaved=False, seed=0, std=1.0,
                 behind=0, with_q=True, pool_std=1.0):
        self.sk, self.n, self.P, self.dtype, self.interleaved = sk, n, P, dtype, interleaved
        rot = D if rot is None else rot
        g = torch.Generator().manual_seed(seed)
        self.bt, self.nb = _q8.block_table(sk, P, seed + 1)
        t = _q8.TORCH[dtype]
        total = sum(n) + behind
        self.q, self.kn, self.vn = ((torch.randn((total, h, D), generator=g) * std).to(t) for h in (H, Hkv, Hkv))
        if not with_q:
            self.q = None
        self.kc, self.ks = _q8.random_pool(self.nb, P, Hkv, D, seed + 2, std=pool_std)
        self.vc, self.vs = _q8.random_pool(self.nb, P, Hkv, D, seed + 3, std=pool_std)
        self.cos, self.sin = _q8.tables(max(sk) + 1, rot) if rot else (None, None)

    def call(self):
        dev = lambda x: None if x is None else x.cuda()  # noqa: E731
        self.got = [dev(x) for x in (self.kc, self.vc, self.ks, self.vs)]
        kc, vc, ks, vs = self.got
        q = dev(self.q)
        self.q_out = binding.kv_append_q8(dev(self.kn), dev(self.vn), _q8.cu(self.n).cuda(), _q8.cu(self.sk).cuda(),
                                          self.bt.cuda(), kc, vc, ks, vs, cos=dev(self.cos), sin=dev(self.sin), q=q,
                                          q_out=None if q is None else torch.full_like(q, 7.0),
                                          interleaved=self.interleaved)
        return self

    def check(self):
        assert binding.device_status() == 0, binding.last_error()
        real = sum(self.n)
        pos = _q8.positions(self.n, self.sk)
        turn = lambda x: (_q8.rotate(x[:real], pos, self.cos, self.sin, self.interleaved) if self.cos is not None  # noqa: E731
                          else (x[:real].double(), torch.zeros_like(x[:real]).double()))
        for new, codes, scale, got_c, got_s in ((turn(self.kn), self.kc, self.ks, self.got[0], self.got[2]),
                                                ((self.vn[:real].double(), torch.zeros_like(self.vn[:real]).double()),
                                                 self.vc, self.vs, self.got[1], self.got[3])):
            want, ws = codes.float().double(), scale.double()
            slack = _q8.append_q8(*new, self.n, self.sk, self.bt, want, ws)
            assert torch.equal(got_s.cpu().double(), ws)
            got = got_c.cpu().float().double()
            assert torch.equal(torch.isnan(got), torch.isnan(want))
            value = torch.nan_to_num(want) * ws[:, None, :, None]
            off = (torch.nan_to_num(got) * ws[:, None, :, None] - value).abs()
            # codes that are given (kept and untouched slots) are exact; a new code is at most one
            # rounding from its value, as the one in 64 bits is
            assert (off <= 2 * slack).all(), float((off - 2 * slack).max())
            differ = (torch.nan_to_num(got) != torch.nan_to_num(want)).double().mean()
            assert differ < 1e-4  # only values within 2^-22 of a tie may land on the other side
        if self.q is not None:
            y, mag = _q8.rotate(self.q[:real], pos, self.cos, self.sin, self.interleaved)
            t = _q8.TORCH[self.dtype]
            tol = torch.finfo(t).eps / 2 * y.abs() * (1 + 2 ** -10) + 3 * 2.0 ** -24 * mag + 2.0 ** -25
            assert ((self.q_out.cpu().double()[:real] - y).abs() <= tol).all()
            assert (self.q_out.cpu()[real:] == 7.0).all()


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_q8_mixed_batch(dtype, interleaved):
    Step([70, 33, 1, 96, 40, 5, 300], [7, 0, 1, 96, 40, 2, 129], dtype=dtype, interleaved=interleaved).call().check()


@pytest.mark.parametrize("D,rot,H,Hkv,P", [(128, 128, 32, 8, 64), (80, 80, 6, 3, 96), (256, 64, 5, 1, 32),
                                           (512, 512, 2, 2, 256), (16, 16, 1, 1, 32), (96, 48, 15, 3, 128)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_q8_head_shapes(D, rot, H, Hkv, P, interleaved):
    Step([513, 1, 257, 90], [100, 1, 30, 90], P=P, H=H, Hkv=Hkv, D=D, rot=rot, interleaved=interleaved,
         seed=D).call().check()


@pytest.mark.parametrize("std", [0.01, 1.0, 50.0])
def test_q8_scale_grows_and_earlier_tokens_are_held_again(std):
    """One new token per sequence: pages keep their scale (small tokens) or grow it."""
    Step(list(range(2, 100, 3)), [1] * 33, std=std, seed=int(std * 100)).call().check()


def test_q8_without_rotation():
    Step([90, 17, 64], [30, 17, 1], D=128, rot=0, with_q=False).call().check()


def test_q8_rows_behind_the_last_sequence_stay():
    Step([40, 9], [8, 9], behind=13).call().check()


def test_q8_not_finite_and_zero_values():
    s = Step([40, 64, 33], [8, 64, 1], D=64, rot=0, with_q=False)
    s.kn[3, 0, 5], s.kn[4, 1, 6], s.vn[2, 0, 1] = float("inf"), float("nan"), float("-inf")
    s.vn[8:40] = 0.0  # a whole page of zeros: the smallest scale
    s.kn[72] = float("nan")  # a single new token without a finite value
    s.call().check()
    assert (s.got[3].cpu()[int(s.bt[1, 0])] == 2.0 ** -100).all()


def test_q8_largest_and_smallest_magnitudes():
    s = Step([64, 32], [64, 32], D=64, rot=0, with_q=False)
    s.kn[:32] = 3.0e38  # bf16, near the type's largest
    s.kn[32:64] = 1.0e-38
    s.vn[0:32] = 448.0  # exactly the largest code at scale 1
    s.vn[32:64] = 450.0
    s.call().check()
    assert (s.got[3].cpu()[int(s.bt[0, 0])] == 1.0).all() and (s.got[3].cpu()[int(s.bt[0, 1])] == 2.0).all()


def test_q8_token_by_token_equals_one_call():
    """A prompt appended token by token holds what one call holds: the same scales, and codes within
    the second rounding of those that fell below the normal range (half a step of 2^-9)."""
    m, P, D = 50, 32, 64
    whole = Step([m], [m], D=D, with_q=False, seed=4).call()
    one = Step([m], [m], D=D, with_q=False, seed=4)
    kc, vc, ks, vs = (x.cuda() for x in (one.kc, one.vc, one.ks, one.vs))
    for i in range(m):
        binding.kv_append_q8(one.kn[i:i + 1].cuda(), one.vn[i:i + 1].cuda(), _q8.cu([1]).cuda(), _q8.cu([i + 1]).cuda(),
                             one.bt.cuda(), kc, vc, ks, vs, cos=one.cos.cuda(), sin=one.sin.cuda())
    assert binding.device_status() == 0
    assert torch.equal(ks, whole.got[2]) and torch.equal(vs, whole.got[3])
    for a, b in ((kc, whole.got[0]), (vc, whole.got[1])):
        a, b = a.float(), b.float()
        assert ((a - b).abs() <= torch.where(b.abs() <= 2.0 ** -6, 2.0 ** -9, 0.0)).all()


def test_q8_same_call_twice_changes_nothing():
    s = Step([70, 33, 5], [7, 1, 5], std=4.0).call()
    first = [x.clone() for x in s.got]
    s.kc, s.vc, s.ks, s.vs = (x.cpu() for x in first)
    s.call()
    for a, b in zip(first, s.got):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def test_q8_strided_caches_and_scales():
    """K and V as halves of one buffer, scales of both in one tensor with the head outermost."""
    sk, n, P, Hkv, D = [70, 33], [40, 33], 32, 2, 64
    ref = Step(sk, n, P=P, Hkv=Hkv, D=D, with_q=False, seed=8)
    both = torch.empty((ref.nb, 2, P, Hkv, D), dtype=torch.float8_e4m3fn, device="cuda")
    both[:, 0], both[:, 1] = ref.kc.cuda(), ref.vc.cuda()
    sc = torch.empty((2, Hkv, ref.nb), device="cuda")
    sc[0], sc[1] = ref.ks.t().cuda(), ref.vs.t().cuda()
    binding.kv_append_q8(ref.kn.cuda(), ref.vn.cuda(), _q8.cu(n).cuda(), _q8.cu(sk).cuda(), ref.bt.cuda(), both[:, 0],
                         both[:, 1], sc[0].t(), sc[1].t(), cos=ref.cos.cuda(), sin=ref.sin.cuda())
    ref.got = [both[:, 0].contiguous(), both[:, 1].contiguous(), sc[0].t().contiguous(), sc[1].t().contiguous()]
    ref.check()


def test_q8_bad_page_is_reported_others_written():
    s = Step([40, 40], [40, 40], with_q=False, seed=9)
    good = s.bt[0, 1].item()
    s.bt[0, 1] = s.nb + 5
    s.call()
    assert binding.STATUS[binding.device_status()] == "PA_ERR_DEVICE_BOUNDS"
    s.bt[0, 1] = good
    got = s.got[0].cpu().view(torch.uint8)
    assert torch.equal(got[good], s.kc.view(torch.uint8)[good])
    for page in (s.bt[0, 0], s.bt[1, 0], s.bt[1, 1]):
        assert not torch.equal(got[int(page)], s.kc.view(torch.uint8)[int(page)])


def test_q8_more_new_tokens_than_keys_is_reported():
    s = Step([8, 3], [8, 3], with_q=False)
    s.sk = [5, 3]
    s.call()
    assert binding.STATUS[binding.device_status()] == "PA_ERR_DEVICE_BOUNDS"
    assert torch.equal(s.got[0].cpu().view(torch.uint8)[int(s.bt[0, 0])], s.kc.view(torch.uint8)[int(s.bt[0, 0])])


def test_q8_captured_and_replayed():
    """A captured append of one token follows the lengths of each replay over a page border."""
    P, D, H = 32, 64, 2
    bt = torch.arange(2, dtype=torch.int32)[None].cuda()
    g = torch.Generator().manual_seed(1)
    x = torch.randn((40, 1, D), generator=g).bfloat16()
    cos, sin = _q8.tables(64, D)
    kc = torch.zeros((2, P, 1, D), device="cuda").to(torch.float8_e4m3fn)
    vc, ks = kc.clone(), torch.zeros((2, 1), device="cuda")
    vs = ks.clone()
    new, keys, now = _q8.cu([1]).cuda(), _q8.cu([1]).cuda(), x[:1].cuda()
    call = lambda: binding.kv_append_q8(now, now, new, keys, bt, kc, vc, ks, vs, cos=cos.cuda(), sin=sin.cuda())  # noqa: E731
    cos, sin = cos.cuda(), sin.cuda()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        call()
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        call()
    want_v, wvs = torch.zeros((2, P, 1, D), dtype=torch.float64), torch.zeros((2, 1), dtype=torch.float64)
    for m in range(1, 41):
        keys[1] = m
        now.copy_(x[m - 1:m])
        graph.replay()
        _q8.append_q8(x[m - 1:m].double(), torch.zeros((1, 1, D)).double(), [1], [m], bt.cpu(), want_v, wvs)
    torch.cuda.synchronize()
    assert binding.device_status() == 0
    assert torch.equal(vs.cpu().double(), wvs)
    assert torch.equal(vc.cpu().float().double(), want_v)

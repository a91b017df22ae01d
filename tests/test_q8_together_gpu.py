"""The 8-bit cache as a server uses it: chunks and single tokens appended to a paged cache, rotated on the
way, and attended, step after step (GPU), against the same run in 64 bits on the values the cache holds; and
the calls' streams, graphs and workspaces."""
import threading

import pytest
import torch

from paged_kv_varlen_flashattention_gb300 import binding
from tests import _q8
from tests.test_q8_attention_gpu import call, inputs, run

pytestmark = pytest.mark.gpu


class Server:
    """Sequences with pages of their own in a shuffled pool; ``step`` appends n[b] tokens to each and attends."""

    def __init__(self, B, pages, P=64, H=8, Hkv=2, D=128, dtype=torch.bfloat16, seed=0):
        g = torch.Generator().manual_seed(seed)
        self.P, self.H, self.Hkv, self.D, self.dtype, self.g = P, H, Hkv, D, dtype, g
        nb = B * pages + 3
        self.bt = torch.randperm(nb, generator=g)[:B * pages].reshape(B, pages).int()
        self.k = torch.full((nb, P, Hkv, D), 0x7F, dtype=torch.uint8).cuda().view(torch.float8_e4m3fn)  # NaN
        self.v = self.k.clone()
        self.ks = torch.full((nb, Hkv), float("nan"), device="cuda")
        self.vs = self.ks.clone()
        self.cos, self.sin = (t.cuda() for t in _q8.tables(pages * P, D))
        self.sk = [0] * B
        self.bt_d = self.bt.cuda()

    def tokens(self, n):
        # a fused projection of q, k and v: strided views of one tensor
        x = torch.randn((sum(n), self.H + 2 * self.Hkv, self.D), generator=self.g).to(self.dtype).cuda()
        return x[:, :self.H], x[:, self.H:self.H + self.Hkv], x[:, self.H + self.Hkv:]

    def step(self, n, wl=-1, **kw):
        q, k, v = self.tokens(n)
        self.sk = [a + b for a, b in zip(self.sk, n)]
        cu_n, cu_k = _q8.cu(n).cuda(), _q8.cu(self.sk).cuda()
        qr = binding.kv_append_q8(k, v, cu_n, cu_k, self.bt_d, self.k, self.v, self.ks, self.vs, cos=self.cos, sin=self.sin,
                                  q=q, **kw)
        out, lse = binding.varlen_fwd_q8(qr, self.k, self.v, self.ks, self.vs, cu_n, cu_k, self.bt_d,
                                         max_seqlen_q=max(n), max_seqlen_k=max(self.sk), window_left=wl, **kw)
        return qr, out, lse, list(n), list(self.sk), wl

    def check(self, result):
        qr, out, lse, n, sk, wl = result
        assert binding.device_status() == 0, binding.last_error()
        kk, vv = (torch.nan_to_num(_q8.values(c.cpu(), torch.nan_to_num(s.cpu()))) for c, s in ((self.k, self.ks),
                                                                                               (self.v, self.vs)))
        args = (_q8.cu(n), _q8.cu(sk), self.bt, self.D ** -0.5, wl, 0, None)
        ref, ref_l = _q8.attention(qr.cpu(), kk, vv, *args)
        mag, _ = _q8.attention(qr.cpu(), kk, vv.abs(), *args)
        # weights within 2^-9 of themselves, what is below them (2^-14 of the largest) on values of at
        # most max |V|, the rounding of out: as in test_q8_attention_gpu
        eps = torch.finfo(self.dtype).eps / 2
        tol = (2.0 ** -9 + 2.0 ** -15) * mag + 2.0 ** -22 * vv.abs().max() * max(sk) + eps * ref.abs() * 1.01 + 1e-30
        assert ((out.cpu().double() - ref).abs() <= tol).all()
        fin = torch.isfinite(ref_l)
        assert ((lse.cpu().double() - ref_l)[fin].abs() <= 2e-5 + 1e-6 * ref_l[fin].abs()).all()


@pytest.mark.parametrize("D,H,Hkv,dtype", [(128, 8, 2, torch.bfloat16), (64, 4, 4, torch.float16), (192, 10, 2, torch.bfloat16)])
def test_serving_run(D, H, Hkv, dtype):
    """A prompt chunk each, a second chunk for some beside single tokens, and ten decode steps that cross pages."""
    s = Server(4, 8, P=64, H=H, Hkv=Hkv, D=D, dtype=dtype, seed=D)
    s.check(s.step([200, 1, 63, 128]))
    s.check(s.step([1, 150, 1, 70], wl=100))
    for i in range(10):
        r = s.step([1, 1, 1, 1])
        if i % 3 == 0:
            s.check(r)


def _decode_step(s):
    """A decode step of fixed shapes, its lengths and tokens in tensors that the host updates."""
    B = len(s.sk)
    x = torch.zeros((B, s.H + 2 * s.Hkv, s.D), dtype=s.dtype, device="cuda")
    q, k, v = x[:, :s.H], x[:, s.H:s.H + s.Hkv], x[:, s.H + s.Hkv:]
    cu_n, cu_k = _q8.cu([1] * B).cuda(), _q8.cu(s.sk).cuda()
    qr = torch.empty((B, s.H, s.D), dtype=s.dtype, device="cuda")
    out, lse = torch.empty_like(qr), torch.empty((s.H, B), device="cuda")
    most = s.bt.shape[1] * s.P

    def one():
        binding.kv_append_q8(k, v, cu_n, cu_k, s.bt_d, s.k, s.v, s.ks, s.vs, cos=s.cos, sin=s.sin, q=q, q_out=qr)
        binding.varlen_fwd_q8(qr, s.k, s.v, s.ks, s.vs, cu_n, cu_k, s.bt_d, max_seqlen_q=1, max_seqlen_k=most, out=out,
                              softmax_lse=lse)

    return x, cu_k, qr, out, lse, one


@pytest.mark.parametrize("B", [3, 70])
def test_captured_decode_steps(B):
    """One capture at the cache's largest length, replayed while the lengths grow; the library's buffers exist
    since a call on the capturing stream before it."""
    s = Server(B, 6, P=32, H=4, Hkv=2, D=128, seed=B)
    s.check(s.step([(37 * b) % 150 + 1 for b in range(B)]))
    st = torch.cuda.Stream()
    x, cu_k, qr, out, lse, one = _decode_step(s)
    keep = [t.clone() for t in (s.k.view(torch.uint8), s.v.view(torch.uint8), s.ks, s.vs)]
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        one()  # warm; it appends over the last token: undone below
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=st):
        one()
    for t, c in zip((s.k.view(torch.uint8), s.v.view(torch.uint8), s.ks, s.vs), keep):
        t.copy_(c)
    for _ in range(4):
        x.copy_(torch.randn(x.shape, generator=s.g).to(s.dtype))
        s.sk = [a + 1 for a in s.sk]
        cu_k.copy_(_q8.cu(s.sk))
        graph.replay()
        torch.cuda.synchronize()
        s.check((qr, out, lse, [1] * B, list(s.sk), -1))


@pytest.mark.parametrize("D", [128, 256])
def test_captured_prompts_share_a_workspace(D):
    """Two captured calls of one stream's workspace, replayed in turn and again: prefill beside decode (the
    side stream's fork and join in the graph), and splits with their combine."""
    st = torch.cuda.Stream()
    runs = []
    for i, (sq, sk) in enumerate((([300, 1, 140], [600, 900, 140]), ([1, 1], [9000, 5000]))):
        x = inputs(sq, sk, H=8, Hkv=2, D=D, P=64, seed=40 + i)
        d = {n: x[n].cuda() for n in ("q", "k", "v", "ks", "vs", "bt")}
        a = (d["q"], d["k"], d["v"], d["ks"], d["vs"], _q8.cu(sq).cuda(), _q8.cu(sk).cuda(), d["bt"])
        kw = dict(max_seqlen_q=max(sq), max_seqlen_k=max(sk), out=torch.empty_like(d["q"]),
                  softmax_lse=torch.empty((8, sum(sq)), device="cuda"))
        want = [t.clone() for t in binding.varlen_fwd_q8(*a, **{**kw, "out": None, "softmax_lse": None})]
        torch.cuda.synchronize()
        with torch.cuda.stream(st):
            binding.varlen_fwd_q8(*a, **kw)
        runs.append((a, kw, want))
    torch.cuda.synchronize()
    graphs = []
    for a, kw, _ in runs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=st):
            binding.varlen_fwd_q8(*a, **kw)
        graphs.append(g)
    for order in ((0, 1), (1, 0), (0, 0, 1)):
        for i in order:
            runs[i][1]["out"].fill_(float("nan"))
            with torch.cuda.stream(st):
                graphs[i].replay()
            torch.cuda.synchronize()
            assert torch.equal(runs[i][1]["out"], runs[i][2][0])
            assert torch.equal(runs[i][1]["softmax_lse"], runs[i][2][1])
    assert binding.device_status() == 0


def test_streams_and_threads():
    """Calls from two threads on streams of their own, each with splits and prefill in its own workspace,
    give what they give alone."""
    cases = [inputs(sq, sk, H=8, Hkv=2, D=128, P=64, seed=60 + i)
             for i, (sq, sk) in enumerate((([300, 1, 40], [900, 7000, 40]), ([1, 1, 1], [3000, 8000, 1])))]
    alone = [call(x) for x in cases]
    torch.cuda.synchronize()
    errors, got = [], [[], []]

    def work(i):
        try:
            st = torch.cuda.Stream()
            with torch.cuda.stream(st):
                for _ in range(8):
                    got[i].append(call(cases[i]))
                st.synchronize()
        except Exception as e:  # noqa: BLE001 - reported below
            errors.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not errors
    for i in range(2):
        for out, lse in got[i]:
            assert torch.equal(out, alone[i][0]) and torch.equal(lse, alone[i][1])


def test_repeats_are_the_same():
    """No atomics order the sums: the same call gives the same bits, whichever items its CTAs took."""
    for sq, sk, D in (([1] * 40, [50 * (i + 1) for i in range(40)], 128), ([500, 300, 1], [900, 300, 4000], 128),
                      ([500, 300, 1], [900, 300, 4000], 256), ([4, 4], [9000, 3000], 256)):
        x = inputs(sq, sk, H=8, Hkv=2, D=D, P=64, seed=len(sq))
        a = call(x)
        for _ in range(3):
            b = call(x)
            assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("B,Hkv,keys,rows", [(1, 1, 300, 1), (4, 2, 700, 1), (16, 8, 3000, 1), (2, 2, 1500, 2), (3, 1, 2000, 4),
                                             (9, 2, 5000, 1)])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_units_shared_by_a_cluster(B, Hkv, keys, rows, dtype):
    """Decode units whose keys a cluster shares, of equal and of ragged lengths (some CTAs of a cluster are left
    without a tile), for every body of the kernel."""
    for G in (1, 3, 4, 7, 16) if B * Hkv < 64 else (1, 7):
        run([rows] * B, [keys] * B, H=G * Hkv, Hkv=Hkv, D=128, P=32, dtype=dtype, seed=B + G)
        run([rows] * B, [max(rows, keys // (b + 1)) if b % 3 != 2 else rows for b in range(B)], H=G * Hkv, Hkv=Hkv, D=80, P=96,
            dtype=dtype, seed=B + G + 1, wl=keys // 2 if G == 3 else -1)


def test_long_offsets():
    """A cache whose byte offsets pass 2^31 (and element offsets of the scales, 2^16 pages): one sequence at
    its far end, written by the append and read by both kernels."""
    P, Hkv, D = 64, 8, 128
    nb = (1 << 31) // (P * Hkv * D) + 40
    k = torch.zeros((nb, P, Hkv, D), dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    v = torch.zeros_like(k)
    ks = torch.zeros((nb, Hkv), device="cuda")
    vs = torch.zeros_like(ks)
    n = 200
    bt = torch.arange(nb - 1, nb - 5, -1).int().reshape(1, 4)
    g = torch.Generator().manual_seed(1)
    kn, vn, q = (torch.randn((n, h, D), generator=g).bfloat16().cuda() for h in (Hkv, Hkv, 2 * Hkv))
    cu = _q8.cu([n]).cuda()
    binding.kv_append_q8(kn, vn, cu, cu, bt.cuda(), k, v, ks, vs)
    out, lse = binding.varlen_fwd_q8(q, k, v, ks, vs, cu, cu, bt.cuda(), max_seqlen_q=n, max_seqlen_k=n)
    last, _ = binding.varlen_fwd_q8(q[-1:], k, v, ks, vs, _q8.cu([1]).cuda(), cu, bt.cuda(), max_seqlen_q=1, max_seqlen_k=n)
    assert binding.device_status() == 0
    sel = bt.flatten().long().cuda()
    kk, vv = (_q8.values(c.view(torch.uint8)[sel].cpu().view(torch.float8_e4m3fn), s[sel].cpu()) for c, s in ((k, ks), (v, vs)))
    # the codes hold the tokens to half a step of e4m3 (a scale of a power of two: subnormals below 2^-6 of it)
    want = kn.cpu().double()
    have = kk.reshape(-1, Hkv, D)[:n]
    step = ks[sel].cpu().double().repeat_interleave(P, 0)[:n, :, None]
    assert ((have - want).abs() <= torch.maximum(want.abs() * 2.0 ** -4, step * 2.0 ** -10)).all()
    ref, _ = _q8.attention(q.cpu(), kk, vv, _q8.cu([n]), _q8.cu([n]), torch.arange(4).int().reshape(1, 4), D ** -0.5, -1, 0, None)
    mag, _ = _q8.attention(q.cpu(), kk, vv.abs(), _q8.cu([n]), _q8.cu([n]), torch.arange(4).int().reshape(1, 4), D ** -0.5, -1, 0,
                           None)
    tol = (2.0 ** -9 + 2.0 ** -15) * mag + 2.0 ** -22 * vv.abs().max() * n + 2.0 ** -8 * ref.abs()
    assert ((out.cpu().double() - ref).abs() <= tol).all()
    assert ((last.cpu().double() - ref[-1:]).abs() <= tol[-1:]).all()


@pytest.mark.parametrize("sq,D", [([1, 1], 128), ([4, 4], 128), ([1, 1], 256), ([300, 200], 256)])
def test_bounded_waits_of_every_kernel(sq, D):
    """Waits that run out (loads withheld): clusters of both bodies, splits of wide heads, the wide prefill.  The
    calls end, report it, and the next call is as it should be."""
    x = inputs(sq, [3000, 900], H=8, Hkv=2, D=D, P=64, seed=5)
    want = call(x)
    torch.cuda.synchronize()
    assert binding.device_status() == 0
    binding.set_wait_limit_ns(20_000_000)
    binding.set_withhold_loads(True)
    try:
        call(x)
        assert binding.STATUS[binding.device_status()] == "PA_ERR_DEVICE_TIMEOUT"
    finally:
        binding.set_withhold_loads(False)
        binding.set_wait_limit_ns(0)
    out, lse = call(x)
    assert binding.device_status() == 0
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])


def test_bad_blocks_in_a_cluster():
    """A block outside the pool in one CTA's share of a unit, and a sequence longer than promised: reported, the
    other sequences as they should be."""
    x = inputs([1, 1, 1], [3000, 2000, 900], H=4, Hkv=1, D=128, P=64, seed=6)
    want = call(x)
    torch.cuda.synchronize()
    good = x["bt"].clone()
    x["bt"][0, 20] = x["k"].shape[0] + 5
    x["bt"][2, 3] = -1
    out, _ = call(x)
    assert binding.STATUS[binding.device_status()] == "PA_ERR_DEVICE_BOUNDS"
    assert torch.equal(out[1], want[0][1])
    x["bt"] = good
    out, _ = call(x, max_sk=2000)
    assert binding.STATUS[binding.device_status()] == "PA_ERR_DEVICE_BOUNDS"
    out, lse = call(x)
    assert binding.device_status() == 0 and torch.equal(out, want[0]) and torch.equal(lse, want[1])


def test_outputs_of_a_call_on_a_given_stream():
    """Outputs that a call allocates come from the memory of the stream it is given, and hold its results."""
    s = Server(2, 4, seed=9)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    r = s.step([100, 1], stream=side)
    side.synchronize()
    s.check(r)
    segments = torch.cuda.memory_snapshot()
    for t in r[:3]:
        own = [g for g in segments if g["address"] <= t.data_ptr() < g["address"] + g["total_size"]]
        assert len(own) == 1 and own[0]["stream"] == side.cuda_stream

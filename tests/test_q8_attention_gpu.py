"""pa_varlen_fwd_q8 on the GPU against attention in 64 bits over the values the cache stands for
(GPU).

Tolerance.  The codes are exact in f16 and the products accumulate in fp32, so a score s (log2
units, |s| <= 64 here) is off by at most 2^-16 for inputs of a few units: 2^-16 ln 2 relative on a
weight.  The weights are rounded for the product with V, at most w each, relative: to f16, w = 2^-11;
in bf16 calls of few rows to two e4m3 terms, of which the first leaves at most half its last place
(2^-4 of the power of two at the weight) and the second half its own (2^-5 of the power of two below
that): w = 2^-9; f16 calls of few rows take three terms, within 2^-11.  A weight below the terms' range
is off by at most half of 2^-13 on the scale where the row's largest weight is 2^8: 2^-22 of the
largest, and the weights sum to at least the largest.  With A = sum_j p_j |V_j| the output before its
own rounding is then off by at most (w + 2^-15) A + 2^-22 sum_j |V_j| over the row's keys, and the
rounding to the type adds eps / 2 of the value (2^-8 bf16, 2^-11 f16) and half a subnormal step.
lse is off by at most 2^-16 from the scores plus fp32 roundings: 2e-5."""
import pytest
import torch

from paged_kv_varlen_flashattention_gb300 import binding
from tests import _q8

pytestmark = pytest.mark.gpu


def inputs(sq, sk, P=32, H=4, Hkv=2, D=64, dtype="bf16", seed=0, kind="pow2", nan_fill=True, q_std=1.0, std=1.0):
    bt, nb = _q8.block_table(sk, P, seed)
    k, ks = _q8.random_pool(nb, P, Hkv, D, seed + 1, kind, std)
    v, vs = _q8.random_pool(nb, P, Hkv, D, seed + 2, kind, std)
    if nan_fill:  # slots no sequence owns, and the scales of blocks no sequence owns
        owned = torch.zeros((nb, P), dtype=torch.bool)
        for b, m in enumerate(sk):
            for p in range((m + P - 1) // P):
                owned[bt[b, p], :min(P, m - p * P)] = True
        for x, s in ((k, ks), (v, vs)):
            x.view(torch.uint8)[~owned] = 0x7F
            s[~owned.any(1)] = float("nan")
    q = (torch.randn((sum(sq), H, D), generator=torch.Generator().manual_seed(seed + 3)) * q_std).to(_q8.TORCH[dtype])
    return dict(q=q, k=k, v=v, ks=ks, vs=vs, bt=bt, sq=sq, sk=sk, dtype=dtype)


def call(x, wl=-1, wr=0, scale=None, slopes=None, max_sq=None, max_sk=None, **kw):
    d = {n: x[n].cuda() for n in ("q", "k", "v", "ks", "vs", "bt")}
    return binding.varlen_fwd_q8(d["q"], d["k"], d["v"], d["ks"], d["vs"], _q8.cu(x["sq"]).cuda(), _q8.cu(x["sk"]).cuda(),
                                 d["bt"], max_seqlen_q=max(x["sq"]) if max_sq is None else max_sq,
                                 max_seqlen_k=max(x["sk"]) if max_sk is None else max_sk, softmax_scale=scale,
                                 window_left=wl, window_right=wr,
                                 alibi_slopes=None if slopes is None else slopes.cuda(), **kw)


def check(x, out, lse, wl=-1, wr=0, scale=None, slopes=None, wide_rows=False):
    """``wide_rows``: q rows of the tensor-core prefill whose columns differ by many powers of two.
    That kernel holds a row of q in e4m3 terms, each element within 2^-10 of a scale on which the
    row's largest is at least 224: within 2^-17.8 of max |q|.  A score is then off by at most ds =
    scale 2^-17.8 max |q| max_j sum_d |k_jd|, a weight by a factor e^(2 ds) after its
    normalisation, lse by ds."""
    assert binding.device_status() == 0, binding.last_error()
    scale = x["q"].shape[-1] ** -0.5 if scale is None else scale
    kk, vv = (torch.nan_to_num(_q8.values(x[a], torch.nan_to_num(x[b]))) for a, b in (("k", "ks"), ("v", "vs")))
    args = (_q8.cu(x["sq"]), _q8.cu(x["sk"]), x["bt"], scale, wl, wr, slopes)
    ref, ref_l = _q8.attention(x["q"], kk, vv, *args)
    mag, _ = _q8.attention(x["q"], kk, vv.abs(), *args)
    t = _q8.TORCH[x["dtype"]]
    w = 2.0 ** -9 if x["dtype"] == "bf16" else 2.0 ** -11
    seq = torch.repeat_interleave(torch.arange(len(x["sq"])), torch.tensor(x["sq"], dtype=torch.long))
    below = torch.stack([vv[x["bt"][b, :(m + vv.shape[1] - 1) // vv.shape[1]].long()].abs().sum((0, 1)) if m else
                         torch.zeros(vv.shape[2:], dtype=torch.float64) for b, m in enumerate(x["sk"])])
    below = below[seq].repeat_interleave(x["q"].shape[1] // vv.shape[2], 1)  # sum |V| of a row's sequence
    tol = (w + 2.0 ** -15) * mag + 2.0 ** -22 * below + torch.finfo(t).eps / 2 * ref.abs() * (1 + 2 ** -8) + \
        torch.finfo(t).smallest_normal * torch.finfo(t).eps / 2
    lse_tol = 2e-5 + 1e-6 * ref_l.abs()
    if wide_rows:
        ds = scale * 2.0 ** -17.8 * x["q"].double().abs().amax(-1) * kk.abs().sum(-1).max()  # (tokens, heads)
        tol = tol + torch.expm1(2 * ds)[..., None] * mag
        lse_tol = lse_tol + ds.t()
    n = sum(x["sq"])
    err = (out.cpu().double()[:n] - ref[:n]).abs()
    assert (err <= tol[:n]).all(), f"{float((err / tol[:n]).max())} of the tolerance"
    got_l = lse.cpu().double()[:, :n]
    assert torch.equal(torch.isneginf(got_l), torch.isneginf(ref_l))
    fin = torch.isfinite(ref_l)
    assert ((got_l - ref_l)[fin].abs() <= lse_tol[fin]).all(), float((got_l - ref_l)[fin].abs().max())


def run(sq, sk, wl=-1, wr=0, scale=None, slopes=None, **kw):
    x = inputs(sq, sk, **kw)
    out, lse = call(x, wl, wr, scale, slopes)
    check(x, out, lse, wl, wr, scale, slopes)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("D,P", [(16, 32), (64, 32), (80, 96), (96, 64), (128, 32), (128, 128), (192, 64), (256, 256),
                                 (320, 32), (512, 64)])
def test_decode_head_dims(D, P, dtype):
    run([1] * 7, [1, 31, 32, 33, 127, 300, 700], D=D, P=P, dtype=dtype, seed=D)


@pytest.mark.parametrize("H,Hkv", [(1, 1), (8, 8), (15, 3), (32, 2), (24, 1), (64, 2)])
@pytest.mark.parametrize("D", [64, 128, 256, 512])
def test_groups_of_query_heads(H, Hkv, D):
    run([1, 1, 2, 1], [5, 260, 140, 77], H=H, Hkv=Hkv, D=D, seed=H)


@pytest.mark.parametrize("D", [64, 128, 256, 512])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_long_queries(D, dtype):
    """Prompts, chunks and single tokens in one call."""
    run([1, 70, 129, 3, 300], [200, 70, 400, 3, 301], D=D, dtype=dtype, seed=D + 1)


@pytest.mark.parametrize("wl,wr", [(0, 0), (20, 0), (-1, -1), (5, 7), (100, -1), (-1, 3)])
@pytest.mark.parametrize("D", [128, 512])
def test_windows(wl, wr, D):
    run([1, 4, 60, 150], [333, 140, 200, 150], wl=wl, wr=wr, D=D, P=64, seed=wl + 200)


def test_rows_without_keys():
    """More queries than keys under a causal mask, no keys at all, no queries."""
    run([5, 3, 0, 1, 64], [2, 0, 40, 1, 9], D=64)
    run([5, 3, 0, 1, 64], [2, 0, 40, 1, 9], D=512)


@pytest.mark.parametrize("kind", ["absmax", "wide"])
@pytest.mark.parametrize("D", [64, 128, 256, 512])
def test_scales_of_other_quantisers(kind, D):
    """Scales that are no powers of two, and pages whose magnitudes span 2^24."""
    x = inputs([1, 1, 33], [500, 90, 260], D=D, kind=kind, seed=5, q_std=0.25)
    if kind == "wide":  # keys of one magnitude, values of many
        x["k"], x["ks"] = _q8.random_pool(x["k"].shape[0], 32, 2, D, 6)
    out, lse = call(x)
    check(x, out, lse)


def test_zero_and_tiny_value_scales():
    """Pages of zeros (the smallest scale, or scale 0) keep their share of the weights."""
    x = inputs([1, 20], [200, 150], D=128, seed=8, nan_fill=False)
    for page, s in ((0, 2.0 ** -100), (2, 0.0)):
        x["v"].view(torch.uint8)[x["bt"][0, page].long()] = 0
        x["vs"][x["bt"][0, page].long()] = s
    out, lse = call(x)
    check(x, out, lse)


def test_bf16_queries_of_any_magnitude():
    """q in bf16 beyond f16's range and far below it."""
    for std, scale in ((3e6, 1e-7), (1e-7, 1e5), (1e30, 1e-31)):
        run([1, 40], [200, 90], D=128, q_std=std, scale=scale)
    run([1, 40], [200, 90], D=512, q_std=3e6, scale=1e-7)


def test_large_scores_keep_their_softmax():
    run([1, 9], [400, 64], D=128, q_std=5.0, scale=0.2)


@pytest.mark.parametrize("scale", [0.0, -0.2])
def test_scales_that_are_not_positive(scale):
    run([1, 50], [100, 60], D=64, scale=scale)


@pytest.mark.parametrize("D", [64, 128, 256, 512])
def test_linear_position_bias(D):
    slopes = torch.exp2(-torch.arange(1, 7).float())
    run([1, 66, 5], [200, 130, 5], H=6, Hkv=2, D=D, slopes=slopes, seed=11)
    run([40, 3], [90, 300], H=6, Hkv=2, D=D, slopes=slopes, wl=30, wr=9, seed=12)


@pytest.mark.parametrize("D", [64, 128, 256, 512])
@pytest.mark.parametrize("tiles", ["1", "2", "3"])
def test_forced_splits(D, tiles, monkeypatch):
    monkeypatch.setenv("PA_SPLIT_TILES", tiles)
    run([1, 1, 2, 1], [700, 1, 130, 513], H=8, D=D, seed=21)
    run([3, 70], [700, 300], H=8, D=D, seed=22)


def test_work_list_of_many_sequences(monkeypatch):
    """The persistent mode: 40 sequences, some split."""
    monkeypatch.setenv("PA_SPLIT_TILES", "2")
    g = torch.Generator().manual_seed(3)
    sk = torch.randint(0, 900, (40,), generator=g).tolist()
    run([1 if m else 0 for m in sk], sk, D=128, H=8, seed=31)
    run([2] * 40, [max(2, m) for m in sk], D=256, H=40, Hkv=2, seed=32)
    run([0] * 39 + [1], [0] * 39 + [600], D=64, seed=33)


@pytest.mark.parametrize("batch", [3, 170])
def test_order_of_many_sequences(batch):
    g = torch.Generator().manual_seed(batch)
    run([1] * batch, torch.randint(1, 200, (batch,), generator=g).tolist(), D=64, H=16, Hkv=8, seed=batch)


def test_sixteen_and_thirty_two_row_units_together():
    run([1, 4, 2, 3, 1], [300, 40, 200, 130, 1], H=16, Hkv=2, D=128)
    run([1, 4, 2, 3, 1], [300, 40, 200, 130, 1], H=16, Hkv=2, D=256)


def test_rows_behind_the_last_sequence_stay():
    x = inputs([1, 40], [100, 60], D=128)
    out = torch.full((41 + 9, 4, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((4, 50), 7.0, device="cuda")
    x["q"] = torch.cat([x["q"], torch.full((9, 4, 128), float("nan"), dtype=torch.bfloat16)])
    call(x, out=out, softmax_lse=lse)
    assert (out[41:] == 7.0).all() and (lse[:, 41:] == 7.0).all()
    x["q"] = x["q"][:41]
    check(x, out[:41], lse[:, :41])


def test_not_a_number_reaches_only_its_readers():
    x = inputs([1, 1], [100, 90], D=128)
    x["v"].view(torch.uint8)[int(x["bt"][0, 1]), 3, 0, 5] = 0x7F
    out, lse = call(x)
    o = out.cpu().float()
    assert torch.isnan(o[0, :2, 5]).all() and torch.isfinite(o[0, 2:]).all() and torch.isfinite(o[1]).all()
    assert torch.isfinite(o[0, :2, :5]).all()
    x = inputs([1, 1], [100, 90], D=128)
    x["k"].view(torch.uint8)[int(x["bt"][1, 0]), 0, 1, 0] = 0xFF
    out, lse = call(x)
    o = out.cpu().float()
    assert torch.isnan(o[1, 2:]).all() and torch.isfinite(o[0]).all() and torch.isfinite(o[1, :2]).all()
    assert torch.isnan(lse.cpu()[2:, 1]).all()


def test_not_a_number_before_the_window_does_not_matter():
    x = inputs([1, 2], [300, 280], D=128, P=64)
    for b, m in ((0, 300), (1, 280)):
        for j in range(0, m - 52):  # keys no query of the sequence attends under a window of 50
            x["v"].view(torch.uint8)[int(x["bt"][b, j // 64]), j % 64] = 0x7F
            x["k"].view(torch.uint8)[int(x["bt"][b, j // 64]), j % 64] = 0x7F
    out, lse = call(x, 50, 0)
    check(x, out, lse, 50, 0)


def test_strided_tensors():
    """q inside a fused projection, the caches as halves of one buffer, scales with the head outermost."""
    x = inputs([1, 35], [200, 90], D=128, H=8, Hkv=2)
    n, nb = 36, x["k"].shape[0]
    rows = torch.zeros((n, 12 * 128), dtype=torch.bfloat16, device="cuda")
    rows[:, :1024] = x["q"].reshape(n, -1).cuda()
    both = torch.stack([x["k"].view(torch.uint8), x["v"].view(torch.uint8)], 1).cuda().view(torch.float8_e4m3fn)
    sc = torch.stack([x["ks"].t(), x["vs"].t()]).contiguous().cuda()
    out = torch.empty((n, 2, 8, 128), dtype=torch.bfloat16, device="cuda")
    _, lse = binding.varlen_fwd_q8(rows[:, :1024].view(n, 8, 128), both[:, 0], both[:, 1], sc[0].t(), sc[1].t(),
                                   _q8.cu([1, 35]).cuda(), _q8.cu([200, 90]).cuda(), x["bt"].cuda(), max_seqlen_q=35,
                                   max_seqlen_k=200, out=out[:, 1])
    check(x, out[:, 1], lse)


def test_physical_placement_does_not_matter():
    x = inputs([1, 40, 3], [500, 90, 200], D=128, nan_fill=False)
    a, la = call(x)
    perm = torch.randperm(x["k"].shape[0], generator=torch.Generator().manual_seed(9))
    y = dict(x)
    for n in ("k", "v"):
        y[n] = torch.empty_like(x[n])
        y[n].view(torch.uint8)[perm] = x[n].view(torch.uint8)
    for n in ("ks", "vs"):
        y[n] = torch.empty_like(x[n])
        y[n][perm] = x[n]
    y["bt"] = torch.where(x["bt"] >= 0, perm.to(torch.int32)[x["bt"].clamp_min(0).long()], x["bt"])
    b, lb = call(y)
    assert torch.equal(a, b) and torch.equal(la, lb)


def test_bad_blocks_are_reported():
    x = inputs([1, 1], [100, 90], D=128)
    x["bt"][0, 1] = x["k"].shape[0] + 3
    call(x)
    assert binding.STATUS[binding.device_status()] == "PA_ERR_DEVICE_BOUNDS"


def test_longer_sequences_than_promised_are_reported():
    x = inputs([1, 2], [100, 90], D=64)
    call(x, max_sk=64)
    assert binding.STATUS[binding.device_status()] == "PA_ERR_DEVICE_BOUNDS"
    call(x, max_sq=1)
    assert binding.STATUS[binding.device_status()] == "PA_ERR_DEVICE_BOUNDS"


def test_too_many_keys_are_refused():
    bt = torch.zeros((1, 1 << 18), dtype=torch.int32, device="cuda")
    k = torch.zeros((2, 64, 1, 64), device="cuda").to(torch.float8_e4m3fn)
    s = torch.ones((2, 1), device="cuda")
    q = torch.zeros((1, 1, 64), dtype=torch.float16, device="cuda")
    with pytest.raises(binding.PaError) as e:
        binding.varlen_fwd_q8(q, k, k, s, s, _q8.cu([1]).cuda(), _q8.cu([1]).cuda(), bt, max_seqlen_q=1,
                              max_seqlen_k=(1 << 24) - 64)
    assert e.value.name == "PA_ERR_UNSUPPORTED"


def test_nothing_to_do():
    e = torch.empty((0, 4, 64), dtype=torch.bfloat16, device="cuda")
    k = torch.zeros((2, 32, 2, 64), device="cuda").to(torch.float8_e4m3fn)
    s = torch.ones((2, 2), device="cuda")
    out, lse = binding.varlen_fwd_q8(e, k, k, s, s, _q8.cu([]).cuda(), _q8.cu([]).cuda(),
                                     torch.zeros((0, 1), dtype=torch.int32, device="cuda"), max_seqlen_q=0, max_seqlen_k=0)
    assert out.shape == (0, 4, 64) and lse.shape == (4, 0)


def test_withheld_loads_time_out():
    x = inputs([1, 1], [100, 90], D=128)
    y = inputs([1, 1], [100, 90], D=512)
    binding.set_wait_limit_ns(20_000_000)
    binding.set_withhold_loads(True)
    try:
        for z in (x, y):
            call(z)
            assert binding.STATUS[binding.device_status()] == "PA_ERR_DEVICE_TIMEOUT"
    finally:
        binding.set_withhold_loads(False)
        binding.set_wait_limit_ns(0)
    for z in (x, y):
        out, lse = call(z)
        check(z, out, lse)

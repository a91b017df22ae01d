"""The tensor-core prefill of pa_varlen_fwd_q8 against attention in 64 bits: item and tile borders of the
persistent kernel (GPU).  Inputs, tolerance and comparison are those of test_q8_attention_gpu."""
import pytest
import torch

from paged_kv_varlen_flashattention_gb300 import binding
from tests.test_q8_attention_gpu import call, check, inputs, run

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _prefill_kernel_takes_small_calls(monkeypatch):
    monkeypatch.setenv("PA_Q8_ROW_TILES", "0")


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("D", [16, 48, 64, 80, 128])
def test_prompts(D, dtype):
    run([33, 64, 129, 257], [33, 64, 129, 257], H=2, Hkv=1, D=D, dtype=dtype, seed=D)


@pytest.mark.parametrize("H,Hkv", [(1, 1), (3, 1), (4, 4), (10, 2), (16, 1), (64, 1)])
def test_group_sizes(H, Hkv):
    """Groups that divide 128 and that leave padding rows, over several tiles."""
    run([90, 40, 300 // (H // Hkv) + 33], [90, 200, 400], H=H, Hkv=Hkv, D=64, seed=H)


@pytest.mark.parametrize("P", [32, 64, 96, 128, 160, 256])
def test_page_sizes(P):
    run([140, 70], [300, 513], D=128, P=P, H=4, Hkv=2, seed=P)


@pytest.mark.parametrize("m", [1, 31, 32, 127, 128, 129, 255, 256, 257, 385])
def test_key_tile_borders(m):
    run([max(1, m // 2), 40], [m, max(40, m)], H=8, Hkv=1, D=128, seed=m)


@pytest.mark.parametrize("wl,wr", [(0, 0), (100, 0), (-1, -1), (127, 128), (300, -1), (-1, 60)])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_windows(wl, wr, dtype):
    run([200, 50, 33], [500, 50, 390], wl=wl, wr=wr, D=128, P=64, dtype=dtype, seed=wl + 301)


def test_items_with_and_without_a_second_tile():
    """Many short sequences: a CTA meets items of one tile and of two in any order, some without keys."""
    g = torch.Generator().manual_seed(7)
    sq = torch.randint(17, 300, (180,), generator=g).tolist()
    sk = [m + int(torch.randint(0, 200, (1,), generator=g)) if i % 11 else 0 for i, m in enumerate(sq)]
    run(sq, sk, H=2, Hkv=1, D=64, seed=7)
    run([s // 2 + 9 for s in sq], [max(0, k - 30) for k in sk], H=4, Hkv=1, D=128, dtype="f16", seed=8)


def test_one_tile_items_follow_each_other():
    """Every item is one query tile and one key tile."""
    run([33] * 400, [33] * 400, H=2, Hkv=1, D=128, seed=9)


@pytest.mark.parametrize("kind", ["absmax", "wide"])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_scales_of_other_quantisers(kind, dtype):
    from tests import _q8
    x = inputs([150, 33], [500, 260], D=128, kind=kind, dtype=dtype, seed=5)
    if kind == "wide":  # keys of one magnitude, values of many
        x["k"], x["ks"] = _q8.random_pool(x["k"].shape[0], 32, 2, 128, 6)
    out, lse = call(x)
    check(x, out, lse)


def test_zero_key_and_value_scales():
    x = inputs([60, 40], [200, 150], D=128, seed=8, nan_fill=False)
    x["v"].view(torch.uint8)[x["bt"][0, 0].long()] = 0
    x["vs"][x["bt"][0, 0].long()] = 0.0
    x["ks"][x["bt"][1, 1].long()] = 0.0
    out, lse = call(x)
    check(x, out, lse)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_query_magnitudes_within_a_row(dtype):
    """Rows whose columns span the type: large columns beside small ones, and rows of zeros."""
    x = inputs([70, 33], [300, 90], D=128, dtype=dtype, seed=3)
    span = torch.exp2(torch.arange(128).float().remainder(13) - 10)
    x["q"] = (x["q"].float() * span).to(x["q"].dtype)
    x["q"][5] = 0.0
    out, lse = call(x, scale=0.2)
    check(x, out, lse, scale=0.2, wide_rows=True)


def test_bf16_queries_of_any_magnitude():
    for std, scale in ((3e6, 1e-7), (1e-7, 1e5), (1e30, 1e-31)):
        run([70, 40], [200, 90], D=128, q_std=std, scale=scale)


def test_rising_scores_raise_the_reference():
    """Every later key tile scores far above the ones before: O is rescaled at every tile."""
    x = inputs([64, 40], [640, 640], D=64, nan_fill=False, seed=4)
    for b in range(2):
        for p in range(20):
            x["ks"][x["bt"][b, p].long()] *= 2.0 ** (p - 14)
    out, lse = call(x)
    check(x, out, lse)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_linear_position_bias(dtype):
    slopes = torch.exp2(-torch.arange(1, 7).float())
    run([70, 66, 130], [200, 130, 130], H=6, Hkv=2, D=128, slopes=slopes, seed=11, dtype=dtype)
    run([40, 33], [90, 300], H=6, Hkv=2, D=64, slopes=slopes, wl=30, wr=9, seed=12, dtype=dtype)


def test_mixed_batch_beside_decode_rows():
    run([1, 70, 1, 4, 200, 1], [900, 300, 1, 513, 200, 64], H=8, Hkv=2, D=128, seed=13)


def test_not_a_number_outside_an_items_keys_does_not_matter():
    """Slots past the sequence and keys before every window hold NaN codes."""
    x = inputs([64, 70], [500, 400], D=128, P=64, H=2, Hkv=1, seed=3)
    for b, (n, m) in enumerate(((64, 500), (70, 400))):
        for j in range(0, m - n - 40):
            for t in ("k", "v"):
                x[t].view(torch.uint8)[int(x["bt"][b, j // 64]), j % 64] = 0x7F
    out, lse = call(x, 40, 0)
    check(x, out, lse, 40, 0)


def test_rows_behind_the_last_sequence_stay():
    x = inputs([60, 40], [100, 60], D=128)
    out = torch.full((109, 4, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((4, 109), 7.0, device="cuda")
    x["q"] = torch.cat([x["q"], torch.full((9, 4, 128), float("nan"), dtype=torch.bfloat16)])
    call(x, out=out, softmax_lse=lse)
    assert (out[100:] == 7.0).all() and (lse[:, 100:] == 7.0).all()
    x["q"] = x["q"][:100]
    check(x, out[:100], lse[:, :100])


def test_bad_blocks_are_reported():
    x = inputs([60, 40], [100, 60], D=128)
    x["bt"][0, 1] = x["k"].shape[0] + 3
    call(x)
    assert binding.STATUS[binding.device_status()] == "PA_ERR_DEVICE_BOUNDS"


def test_withheld_loads_time_out():
    x = inputs([60, 40], [100, 60], D=128)
    binding.set_wait_limit_ns(20_000_000)
    binding.set_withhold_loads(True)
    try:
        call(x)
        assert binding.STATUS[binding.device_status()] == "PA_ERR_DEVICE_TIMEOUT"
    finally:
        binding.set_withhold_loads(False)
        binding.set_wait_limit_ns(0)
    out, lse = call(x)
    check(x, out, lse)


def test_row_tiles_without_the_tensor_core_kernel(monkeypatch):
    """The same rows on the split-KV kernel (scale <= 0 keeps them there) against the tensor-core one."""
    run([70, 129], [300, 129], D=128, scale=-0.1, seed=17)


@pytest.mark.parametrize("alibi", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_small_calls_on_row_tiles(alibi, dtype, monkeypatch):
    """Calls of few row tiles take the split-KV kernel: one sequence beside another, a group that does not
    divide a tile, and the first sizes past the rule."""
    monkeypatch.delenv("PA_Q8_ROW_TILES")
    slopes = torch.exp2(-torch.arange(1, 11).float()) if alibi else None
    for sq, sk in ([64], [64]), ([256], [300]), ([33, 1, 7], [500, 512, 0]), ([100], [513]), ([400, 90], [400, 900]):
        run(sq, sk, H=10, Hkv=2, D=96, P=96, dtype=dtype, slopes=slopes, seed=sum(sq))


@pytest.mark.parametrize("wl,wr", [(-1, 0), (-1, -1), (200, 100), (0, 300)])
def test_bias_over_many_tiles(wl, wr):
    """Keys on one side of a query's position and on both, over tiles taken from the nearest on."""
    run([300, 140], [1500, 333], H=10, Hkv=2, D=128, P=64, wl=wl, wr=wr,
        slopes=torch.exp2(-torch.arange(1, 11).float()), seed=wl + 7)
    run([260], [2300], H=4, Hkv=4, D=64, P=32, wl=wl, wr=wr, slopes=torch.tensor([1.0, 0.1, 0.01, 0.0]),
        dtype="f16", seed=wl + 8)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("D", [144, 192, 208, 256])
def test_wide_prompts(D, dtype):
    run([33, 64, 129, 257], [33, 64, 129, 257], H=2, Hkv=1, D=D, dtype=dtype, seed=D)


@pytest.mark.parametrize("H,Hkv", [(1, 1), (3, 1), (4, 4), (10, 2), (64, 1)])
def test_wide_group_sizes(H, Hkv):
    run([90, 40, 300 // (H // Hkv) + 33], [90, 200, 400], H=H, Hkv=Hkv, D=256, seed=H)


@pytest.mark.parametrize("m", [1, 31, 32, 63, 64, 65, 127, 128, 129, 193])
def test_wide_key_tile_borders(m):
    """One, two and three key tiles, and a last one that is not full."""
    run([max(1, m // 2), 40], [m, max(40, m)], H=8, Hkv=1, D=256, seed=m)


@pytest.mark.parametrize("wl,wr,slopes", [(0, 0, False), (100, 0, True), (-1, -1, True), (63, 64, False), (300, -1, True),
                                          (-1, 60, False)])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_wide_windows(wl, wr, slopes, dtype):
    run([200, 50, 33], [500, 50, 390], wl=wl, wr=wr, H=4, Hkv=2, D=192, P=96, dtype=dtype, seed=wl + 301,
        slopes=torch.tensor([1.0, 0.1, 0.01, 0.0]) if slopes else None)


@pytest.mark.parametrize("P", [32, 64, 96, 256])
def test_wide_page_sizes(P):
    run([140, 70], [300, 1313], D=256, P=P, H=4, Hkv=2, seed=P, kind="absmax")


def test_wide_items_follow_each_other():
    """Many short items on every CTA, some without keys, one and several key tiles in any order; rows of
    large scores late in a sequence, which raise the reference."""
    g = torch.Generator().manual_seed(17)
    sq = torch.randint(17, 200, (230,), generator=g).tolist()
    sk = [m + int(torch.randint(0, 200, (1,), generator=g)) if i % 11 else 0 for i, m in enumerate(sq)]
    run(sq, sk, H=2, Hkv=1, D=256, seed=7, q_std=4.0)
    run([s // 2 + 9 for s in sq], [max(0, k - 30) for k in sk], H=4, Hkv=1, D=192, dtype="f16", seed=8)

"""Host-side refusals of the rotated append and the 8-bit calls (no GPU, no CUDA call), and the
plain 64-bit implementations that the GPU tests compare with."""
import pytest
import torch

from paged_kv_varlen_flashattention_gb300 import binding
from tests import _q8
from tests.test_validation import desc

CODES = {v: k for k, v in binding.STATUS.items()}
BF, F32, I32, E4 = binding.PA_BF16, binding.PA_F32, binding.PA_I32, binding.PA_E4M3


def rope(**over):
    d = dict(q=desc([8, 4, 64], BF), k_new=desc([8, 2, 64], BF), v_new=desc([8, 2, 64], BF), cos=desc([50, 32], F32),
             sin=desc([50, 32], F32), cu_new=desc([3], I32), cu_k=desc([3], I32), bt=desc([2, 3], I32),
             k=desc([6, 32, 2, 64], BF), v=desc([6, 32, 2, 64], BF), q_out=desc([8, 4, 64], BF))
    P = over.pop("P", 32)
    d.update(over)
    return binding.kv_append_rope_check(list(d.values()), P)


def q8(**over):
    d = dict(q=desc([8, 4, 64], BF), k_new=desc([8, 2, 64], BF), v_new=desc([8, 2, 64], BF), cos=desc([50, 32], F32),
             sin=desc([50, 32], F32), cu_new=desc([3], I32), cu_k=desc([3], I32), bt=desc([2, 3], I32),
             k=desc([6, 32, 2, 64], E4), v=desc([6, 32, 2, 64], E4), ks=desc([6, 2], F32), vs=desc([6, 2], F32),
             q_out=desc([8, 4, 64], BF))
    P = over.pop("P", 32)
    d.update(over)
    return binding.kv_append_q8_check(list(d.values()), P)


COMMON = [
    ("PA_ERR_ARG", dict(k_new=None)),
    ("PA_ERR_ARG", dict(sin=None)),
    ("PA_ERR_ARG", dict(q_out=None)),
    ("PA_ERR_ARG", dict(bt=None)),
    ("PA_ERR_RANK", dict(k_new=desc([8, 128], BF))),
    ("PA_ERR_RANK", dict(cos=desc([32], F32), sin=desc([32], F32))),
    ("PA_ERR_RANK", dict(q=desc([8, 256], BF))),
    ("PA_ERR_NONCONTIG", dict(cos=desc([50, 32], F32, [64, 2]))),
    ("PA_ERR_NONCONTIG", dict(q=desc([8, 4, 64], BF, [512, 128, 2]))),
    ("PA_ERR_SHAPE", dict(sin=desc([49, 32], F32))),
    ("PA_ERR_SHAPE", dict(cos=desc([50, 40], F32), sin=desc([50, 40], F32))),
    ("PA_ERR_SHAPE", dict(cos=desc([50, 0], F32), sin=desc([50, 0], F32))),
    ("PA_ERR_SHAPE", dict(q=desc([7, 4, 64], BF), q_out=desc([7, 4, 64], BF))),
    ("PA_ERR_SHAPE", dict(q_out=desc([8, 5, 64], BF))),
    ("PA_ERR_ARG", dict(cos=desc([50, 32], BF), sin=desc([50, 32], BF))),
    ("PA_ERR_ARG", dict(q=desc([8, 4, 64], binding.PA_F16))),
    ("PA_ERR_UNSUPPORTED", dict(cos=desc([50, 20], F32), sin=desc([50, 20], F32))),
    ("PA_ERR_UNSUPPORTED", dict(cos=desc([50, 32], F32, [34, 1]))),
    ("PA_ERR_UNSUPPORTED", dict(sin=desc([50, 32], F32, None, 0x100004))),
    ("PA_ERR_UNSUPPORTED", dict(q=desc([8, 4, 64], BF, [260, 64, 1]))),
    ("PA_ERR_UNSUPPORTED", dict(q_out=desc([8, 4, 64], BF, None, 0x100008))),
    ("PA_ERR_PAGE_UNSET", dict(P=0)),
    ("PA_ERR_PAGE_MISMATCH", dict(P=64)),
]


@pytest.mark.parametrize("call", [rope, q8])
def test_append_well_formed(call):
    assert call() == 0
    assert call(q=None, q_out=None) == 0
    assert call(cos=desc([50, 16], F32), sin=desc([50, 16], F32)) == 0  # part of the columns
    assert call(q=desc([8, 3, 64], BF, [1024, 64, 1]), q_out=desc([8, 3, 64], BF)) == 0


@pytest.mark.parametrize("call", [rope, q8])
@pytest.mark.parametrize("case", range(len(COMMON)))
def test_append_refusals(call, case):
    name, over = COMMON[case]
    assert binding.STATUS[call(**dict(over))] == name
    assert binding.last_error()


def test_rope_needs_tables():
    assert rope(cos=None, sin=None) == CODES["PA_ERR_ARG"]


def test_rope_refuses_an_8_bit_cache():
    assert rope(k=desc([6, 32, 2, 64], E4), v=desc([6, 32, 2, 64], E4)) == CODES["PA_ERR_UNSUPPORTED"]


@pytest.mark.parametrize("name,over", [
    ("PA_ERR_ARG", dict(cos=None, sin=None)),  # q without tables
    ("PA_ERR_ARG", dict(ks=None)),
    ("PA_ERR_ARG", dict(k=desc([6, 32, 2, 64], BF))),
    ("PA_ERR_ARG", dict(v=desc([6, 32, 2, 64], BF))),
    ("PA_ERR_RANK", dict(ks=desc([6], F32))),
    ("PA_ERR_SHAPE", dict(vs=desc([6, 4], F32))),
    ("PA_ERR_SHAPE", dict(ks=desc([5, 2], F32))),
    ("PA_ERR_ARG", dict(ks=desc([6, 2], BF))),
    ("PA_ERR_UNSUPPORTED", dict(ks=desc([6, 2], F32, [0, 1]))),
    ("PA_ERR_UNSUPPORTED", dict(k=desc([6, 32, 2, 64], E4, [4104, 128, 64, 1]), v=desc([6, 32, 2, 64], E4, [4104, 128, 64, 1]))),
    ("PA_ERR_UNSUPPORTED", dict(k_new=desc([8, 2, 72], BF), v_new=desc([8, 2, 72], BF), q=None, q_out=None,
                                k=desc([6, 32, 2, 72], E4), v=desc([6, 32, 2, 72], E4))),
    ("PA_ERR_UNSUPPORTED", dict(k_new=desc([8, 2, 64], F32), v_new=desc([8, 2, 64], F32))),
])
def test_q8_append_refusals(name, over):
    assert binding.STATUS[q8(**over)] == name


def test_q8_append_without_rotation():
    assert q8(cos=None, sin=None, q=None, q_out=None) == 0


def test_q8_append_head_major_scales():
    assert q8(ks=desc([6, 2], F32, [1, 6]), vs=desc([6, 2], F32, [1, 6])) == 0


def attend(**over):
    d = dict(q=desc([8, 4, 64], BF), k=desc([6, 32, 2, 64], E4), v=desc([6, 32, 2, 64], E4), ks=desc([6, 2], F32),
             vs=desc([6, 2], F32), cu_q=desc([3], I32), cu_k=desc([3], I32), bt=desc([2, 3], I32), alibi=None,
             out=desc([8, 4, 64], BF), lse=desc([4, 8], F32))
    P, sk, D, H, scale = (over.pop(k, v) for k, v in (("P", 32), ("sk", 96), ("D", 64), ("H", 4), ("scale", 0.125)))
    d.update(over)
    return binding.varlen_check_q8(list(d.values()), 5, sk, H, 2, D, P, scale)


def test_q8_attention_well_formed():
    assert attend() == 0
    assert attend(alibi=desc([4], F32)) == 0
    assert attend(ks=desc([6, 2], F32, [1, 6])) == 0


@pytest.mark.parametrize("name,over", [
    ("PA_ERR_ARG", dict(bt=None)),  # always paged
    ("PA_ERR_ARG", dict(q=None)),
    ("PA_ERR_ARG", dict(vs=None)),
    ("PA_ERR_RANK", dict(q=desc([8, 256], BF))),
    ("PA_ERR_RANK_PAGED", dict(k=desc([192, 2, 64], E4))),
    ("PA_ERR_NONCONTIG", dict(k=desc([6, 32, 2, 64], E4, [8192, 256, 128, 2]))),
    ("PA_ERR_SHAPE", dict(v=desc([7, 32, 2, 64], E4))),
    ("PA_ERR_PAGE_UNSET", dict(P=0)),
    ("PA_ERR_PAGE_MISMATCH", dict(P=64)),
    ("PA_ERR_PAGE_MULT32", dict(k=desc([6, 48, 2, 64], E4), v=desc([6, 48, 2, 64], E4), P=48)),
    ("PA_ERR_SHAPE", dict(alibi=desc([5], F32))),
    ("PA_ERR_UNSUPPORTED", dict(q=desc([8, 4, 64], F32))),
    ("PA_ERR_ARG", dict(k=desc([6, 32, 2, 64], BF))),
    ("PA_ERR_ARG", dict(v=desc([6, 32, 2, 64], BF))),
    ("PA_ERR_ARG", dict(out=desc([8, 4, 64], binding.PA_F16))),
    ("PA_ERR_RANK", dict(ks=desc([12], F32))),
    ("PA_ERR_SHAPE", dict(vs=desc([6, 3], F32))),
    ("PA_ERR_ARG", dict(vs=desc([6, 2], BF))),
    ("PA_ERR_ARG", dict(sk=97)),  # the table is too narrow
    ("PA_ERR_ARG", dict(H=8)),
    ("PA_ERR_ARG", dict(scale=float("nan"))),
    ("PA_ERR_UNSUPPORTED", dict(k=desc([6, 32, 2, 64], E4, [4104, 128, 64, 1]), v=desc([6, 32, 2, 64], E4, [4104, 128, 64, 1]))),
    ("PA_ERR_UNSUPPORTED", dict(q=desc([8, 4, 72], BF), out=desc([8, 4, 72], BF), k=desc([6, 32, 2, 72], E4),
                                v=desc([6, 32, 2, 72], E4), D=72)),
    ("PA_ERR_UNSUPPORTED", dict(k=desc([6, 32, 2, 64], E4, None, 0x100008))),
])
def test_q8_attention_refusals(name, over):
    assert binding.STATUS[attend(**over)] == name
    assert binding.last_error()


# ---- the plain implementations themselves ----

def test_plain_e4m3_is_torchs():
    """Every e4m3 value, and the middle between neighbours, rounds as torch's cast does."""
    v = torch.arange(0, 127, dtype=torch.uint8).view(torch.float8_e4m3fn).double()
    mid = (v[:-1] + v[1:]) / 2
    x = torch.cat([v, mid, mid * (1 + 2.0 ** -20), mid * (1 - 2.0 ** -20)])
    x = torch.cat([x, -x])
    assert torch.equal(_q8.e4m3(x), x.float().to(torch.float8_e4m3fn).double())


def test_plain_scale_is_the_least_power_of_two():
    for a in (1e-40, 2.0 ** -100, 447.9, 448.0, 448.1, 3.5, 3.4999, 3.5001, 1.0, 3e38):
        s = _q8.pow2_scale(a)
        assert a <= 448 * s and (a > 448 * s / 2 or s == 2.0 ** -100)
    assert _q8.pow2_scale(0.0) == 2.0 ** -100


def test_plain_rotation_is_a_complex_product():
    x = torch.randn((5, 3, 16), dtype=torch.float64)
    cos, sin = _q8.tables(9, 16)
    pos = torch.tensor([0, 3, 8, 1, 1])
    w = torch.complex(cos[pos].double(), sin[pos].double())[:, None]
    y = torch.view_as_real(torch.view_as_complex(x.reshape(5, 3, 8, 2)) * w).reshape(5, 3, 16)
    assert torch.allclose(_q8.rotate(x, pos, cos, sin, True)[0], y, atol=1e-15)
    y = torch.complex(x[..., :8], x[..., 8:]) * w
    assert torch.allclose(_q8.rotate(x, pos, cos, sin, False)[0], torch.cat((y.real, y.imag), -1), atol=1e-15)


def test_plain_attention_is_torchs():
    g = torch.Generator().manual_seed(2)
    sq, sk, P, H, Hkv, D = [3, 7], [40, 7], 32, 4, 2, 16
    bt, nb = _q8.block_table(sk, P, 3)
    k, v = (torch.randn((nb, P, Hkv, D), generator=g, dtype=torch.float64) for _ in range(2))
    q = torch.randn((10, H, D), generator=g, dtype=torch.float64)
    out, lse = _q8.attention(q, k, v, _q8.cu(sq), _q8.cu(sk), bt, 0.3, -1, 0)
    at = 0
    for b, (n, m) in enumerate(zip(sq, sk)):
        used = bt[b, :(m + P - 1) // P].long()
        kk = k[used].reshape(-1, Hkv, D)[:m].repeat_interleave(2, 1).permute(1, 0, 2)
        vv = v[used].reshape(-1, Hkv, D)[:m].repeat_interleave(2, 1).permute(1, 0, 2)
        mask = torch.ones((n, m), dtype=torch.bool).tril(m - n)
        o = torch.nn.functional.scaled_dot_product_attention(q[at:at + n].permute(1, 0, 2), kk, vv, attn_mask=mask,
                                                             scale=0.3)
        assert torch.allclose(out[at:at + n].permute(1, 0, 2), o, atol=1e-12)
        at += n


def test_tensors_as_descriptors():
    """The binding's module: address, type, sizes and strides of views, None, ranks and types without a code, and
    the outputs it allocates."""
    import torch
    binding._bind_runtime()
    m = binding._runtime[3]
    x = torch.zeros(3, 4, 8, dtype=torch.bfloat16)[1:, ::2]
    types = {torch.float16: 0, torch.bfloat16: 1, torch.float32: 2, torch.int32: 3, torch.float8_e4m3fn: 4, torch.int64: -1}
    buf, *at = m.pack(x, None, *[torch.empty(2, 3, dtype=t) for t in types], torch.zeros(1, 1, 1, 1, 1))
    d = [a if a is None else binding.PaTensor.from_address(a) for a in at]
    assert (d[0].data, d[0].dtype, d[0].ndim) == (x.data_ptr(), 1, 3)
    assert list(d[0].shape) == [2, 2, 8, 0] and list(d[0].stride) == [32, 16, 1, 0]
    assert d[1] is None and [e.dtype for e in d[2:8]] == list(types.values()) and d[8].ndim == 5
    assert len(buf) == 80 * len(d)
    out, lse = m.empty_like(x), m.empty_lse(x)
    assert out.shape == x.shape and out.is_contiguous() and out.dtype == x.dtype
    assert lse.shape == (2, 2) and lse.dtype == torch.float32 and m.empty_lse(torch.empty(3)).numel() == 0
    for f in (m.pack, m.empty_like, m.empty_lse):
        with pytest.raises(TypeError):
            f(3)
    with pytest.raises(RuntimeError):
        m.pack(torch.zeros(2, 2).to_sparse())

"""GPU test of the precision that pa.decode_kv8's softmax weights have where they
meet the values: two fp16 parts, for bf16 outputs one of 11 bits, over each row
tile and plan."""
import math

import pytest
import torch

import cache_reference as cref
import paged_kv_attention_08_gb300 as pa
import step_reference as ref

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
E4M3 = torch.float8_e4m3fn


@pytest.mark.parametrize("dtype,out_dtype,part", [
    (torch.float16, torch.float16, 2.0 ** -16), (torch.bfloat16, torch.float32, 2.0 ** -16),
    (torch.bfloat16, torch.bfloat16, 2.0 ** -11)])
@pytest.mark.parametrize("H,Hkv,D,bs", [(4, 1, 64, 16), (16, 1, 64, 32), (32, 8, 128, 16),
                                        (16, 1, 128, 32), (8, 2, 256, 16), (16, 1, 256, 32)])
@pytest.mark.parametrize("Q,T", [(1, 9), (4, 41), (1, 700), (2, 9100)])
def test_weights_keep_their_bits(Q, T, H, Hkv, D, bs, dtype, out_dtype, part):
    """A score is one product (the query's other elements are 0): exact but for its
    scalings and the exponential.  What is left of an output's error besides its own
    rounding is the weights': in numerator and normaliser T sums of 2^-23 (twice where
    pieces are joined) and exponentials of arguments up to 2^4, four times rounded; and
    the part that a weight loses on the way to the values, in the numerator."""
    table, pool = ref.tables([T], bs, T)
    g = torch.Generator().manual_seed(T + D)
    kc = torch.zeros(pool, bs, Hkv, D).to(E4M3)
    kc[..., 5] = torch.randn(pool, bs, Hkv, generator=g).to(E4M3)
    vc = torch.randn(pool, bs, Hkv, D, generator=g).to(E4M3)
    one = torch.ones(pool, Hkv)
    q = torch.zeros(1, Q, H, D)
    q[..., 5] = 1 + torch.arange(H) / 128
    q = q.to(dtype)
    lens = torch.tensor([T], dtype=torch.int32)
    scale = 1.25
    k, v = cref.values8(kc, one), cref.values8(vc, one)
    want = cref.attention(q, k, v, table, lens, scale)
    mean = cref.attention(q, k, v.abs(), table, lens, scale)
    out = torch.full(q.shape, math.nan, dtype=out_dtype, device=DEV)
    pa.decode_kv8(out, *(x.to(DEV) for x in (q, kc, vc, one, one, table, lens)), scale, T)
    torch.cuda.synchronize()
    assert pa.device_error() == 0
    own = (2 * T + 2) * 2.0 ** -23 + 4 * 0.6932 * 2.0 ** -20
    slack = (2 * own + part) * mean + 2.0 ** -26
    err = (out.cpu().double() - want).abs()
    err -= slack + torch.finfo(out_dtype).eps / 2 * (want.abs() + slack)
    assert err.max().item() <= 0

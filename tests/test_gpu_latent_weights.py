"""GPU test of the precision that pa.decode_latent's softmax weights have where they
meet the values: bf16 ones in two parts (at latent_dim 512 with more than 32 rows in
one of 8 bits), fp16 ones in one of 11 bits, in the row tiles of every size."""
import math

import pytest
import torch

import paged_kv_attention_08_gb300 as pa
import step_reference as ref

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
P = 64


@pytest.mark.parametrize("dtype,part", [(torch.bfloat16, 2.0 ** -16), (torch.float16, 2.0 ** -11)])
@pytest.mark.parametrize("H", [16, 20, 64, 130])
@pytest.mark.parametrize("R", [128, 256, 512])
@pytest.mark.parametrize("T", [9, 41, 700])
def test_weights_keep_their_bits(T, R, H, dtype, part):
    """A score is one product of the positional part (the query's other elements are
    0): exact but for its two scalings and the exponential.  What is left of an
    output's error besides its own rounding is the weights': in numerator and
    normaliser T sums of 2^-23 and an exponential's 2^-22 with an argument of up to
    2^4, three times rounded; and the part that a weight loses on the way to the values."""
    if dtype == torch.bfloat16 and R == 512 and H > 32:
        part = 2.0 ** -8
    table, pool = ref.tables([T], 32, T)
    cache = ref.normal((pool, 32, R + P), dtype, T + 1)
    cache[..., R:] = 0
    cache[..., R] = ref.normal((pool, 32), dtype, T + 2)
    q = torch.zeros(1, 1, H, R + P, dtype=dtype)
    q[..., R] = 1 + torch.arange(H) / 256
    q = q.to(dtype)
    rows, _ = ref._rows(cache.unsqueeze(2), table[0], T, 0)
    p = torch.softmax(q[0, 0].double() @ rows.T * 1.25, 1)
    want, mean = p @ rows[:, :R], p @ rows[:, :R].abs()
    out = torch.full((1, 1, H, R), math.nan, dtype=dtype, device=DEV)
    pa.decode_latent(out, q.to(DEV), cache.to(DEV), table.to(DEV),
                     torch.tensor([T], dtype=torch.int32, device=DEV), 1.25, T)
    torch.cuda.synchronize()
    assert pa.device_error() == 0
    one = (T + 2) * 2.0 ** -23 + 3 * 0.6932 * 2.0 ** -20
    # (a part: of each weight, in the numerator and, where the normaliser sums the rounded ones, there)
    slack = (2 * one + 2 * part) * mean + 2.0 ** -26
    err = (out[0, 0].cpu().double() - want).abs()
    err -= slack + torch.finfo(dtype).eps / 2 * (want.abs() + slack)
    assert err.max().item() <= 0

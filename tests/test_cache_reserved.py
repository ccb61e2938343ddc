"""CPU test: a latent shape whose reserved word is not 0 is refused by every entry
point that takes one, before anything else is looked at."""
import ctypes

import pytest

import paged_kv_attention_08_gb300 as pa
from test_cache_refusals import append_latent, decode_latent, latent, latent_rope, lib  # noqa: F401


@pytest.mark.parametrize("word", [1, -1, 1 << 30])
def test_a_reserved_word_is_refused(lib, word):  # noqa: F811
    s = latent(reserved=word, batch=0)           # (an empty batch reaches no launch)
    nothing = {i: None for i in range(9)}
    assert append_latent(lib, s, latent_rope(), nothing) == 1
    assert decode_latent(lib, s, {i: None for i in range(5)}) == 1
    assert lib.pa_workspace_size_latent(ctypes.byref(latent(reserved=word)), 1, 100) == 0
    assert append_latent(lib, latent(batch=0), latent_rope(), nothing) == 0
    assert pa._LatentShape().reserved == 0

"""Refusals of the 4-bit history cache, without a GPU: every argument check comes before any CUDA call, so the pointers
here are never followed."""
import pytest

P = 1 << 20      # an aligned address that nothing follows


@pytest.fixture(scope="module")
def zg():
    import __graft_entry__
    __graft_entry__.build()
    import generative_recommendation_constrained_gb300 as zg
    return zg


def cache(zg, **kw):
    a = dict(fmt=zg.ZG_KV_E2M1, n_blocks=8, heads=2, block_tokens=16, dim=64, k_codes=P, v_codes=P, k_scale=P, v_scale=P)
    a.update(kw)
    return zg.make_kv_cache(**a)


def refused(zg, status, words, f, *a, **kw):
    with pytest.raises(zg.ZgError) as e:
        f(*a, **kw)
    assert e.value.status == status and words in str(e.value), str(e.value)


@pytest.mark.parametrize("kw, status, words", [(dict(fmt=3), 1, "format"), (dict(dim=80), 4, "dim"), (dict(k_scale=P + 4), 1, "16-byte"),
                                               (dict(v_scale=P + 8), 1, "16-byte"), (dict(v_codes=P + 8), 1, "16-byte"),
                                               (dict(k_scale=None), 1, "NULL"), (dict(block_tokens=8), 1, "block_tokens")])
def test_bad_caches(zg, kw, status, words):
    c, r = cache(zg, **kw), zg.make_rows(P, zg.ZG_BF16, 256, 128, 64)
    refused(zg, status, words, zg.zg_kv_append, c, None, r, r, None, None, 0, P, 4, P, None, 1, 1)
    refused(zg, status, words, zg.zg_kv_read, c, P, 4, P, None, 1, 1, r, r)
    refused(zg, status, words, zg.zg_kv_attention, c, P, 4, P, None, r, r, None, 1, 1, 2, 1.0, False, P, 1 << 30)
    refused(zg, status, words, zg.zg_kv_attention_workspace_size, c, 4, 1, 1, 2)


def test_append_refusals(zg):
    c, r, n = cache(zg), zg.make_rows(P, zg.ZG_BF16, 256, 128, 64), zg.make_norm_rope(True, 1e-6, None, None, 64, False, 1e4)
    f = zg.zg_kv_append
    refused(zg, 1, "start", f, c, n, r, r, None, None, 0, P, 4, None, None, 1, 1)
    refused(zg, 1, "v must", f, c, n, r, zg.make_rows(P, zg.ZG_F16, 256, 128, 64), None, None, 0, P, 4, P, None, 1, 1)
    refused(zg, 1, "without a norm_rope", f, c, None, r, r, r, r, 2, P, 4, P, None, 1, 1)
    refused(zg, 4, "tokens", f, c, n, r, r, None, None, 0, P, 4, P, None, 2 ** 31 - 1, 2 ** 31 - 1)
    refused(zg, 4, "CTAs", f, c, n, r, r, None, None, 0, P, 4, P, None, 2 ** 20, 2 ** 18)
    f(c, n, r, r, None, None, 0, P, 4, P, None, 0, 1)
    f(c, n, r, r, None, None, 0, P, 4, P, None, 1, 0)

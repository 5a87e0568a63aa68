"""Refusals of the prompt attention, without a GPU: every argument check comes before any CUDA call."""
import pytest

P = 1 << 20      # an aligned address that nothing follows


@pytest.fixture(scope="module")
def zg():
    import __graft_entry__
    __graft_entry__.build()
    import generative_recommendation_constrained_gb300 as zg
    return zg


def test_refusals(zg):
    def rows(data=P, dtype=zg.ZG_BF16, st=256, sh=64):
        return zg.make_rows(data, dtype, 0, st, sh)

    r = rows()
    ok = dict(q=r, k=r, v=r, out=r, lse=None, starts=P, B=1, T=8, Hq=4, Hk=2, dim=64, scale=0.125, causal=True)

    def no(status, words, **kw):
        with pytest.raises(zg.ZgError) as e:
            zg.zg_prompt_attention(**{**ok, **kw})
        assert e.value.status == status and words in str(e.value), str(e.value)

    no(4, "dim", dim=80)
    no(1, "B and T", B=-1)
    no(1, "B and T", T=-1)
    no(1, "Hq", Hq=3)
    no(1, "Hq", Hk=0)
    no(1, "Hq", Hq=2048)
    no(1, "2^31", T=2 ** 29)
    no(1, "scale", scale=0.0)
    no(1, "scale", scale=float("nan"))
    no(1, "q is NULL", q=None)
    no(4, "ZG_BF16 or ZG_F16", q=rows(dtype=zg.ZG_F32))
    no(1, "v must", v=rows(dtype=zg.ZG_F16))
    no(1, "out strides", out=rows(st=130))
    no(1, "16-byte", k=rows(data=P + 8))
    no(1, "multiples of 8", v=rows(st=260))
    no(1, "multiples of 8", k=rows(sh=68))
    no(1, "starts", starts=None)
    no(1, "starts", starts=P + 2)
    no(1, "lse", lse=P + 2)
    zg.zg_prompt_attention(**{**ok, "B": 0, "q": None})
    zg.zg_prompt_attention(**{**ok, "T": 0, "q": None})

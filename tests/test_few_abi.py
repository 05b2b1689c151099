"""CPU checks of the few-token layer's entry points: refusals and argument errors come before any
launch."""
import ctypes as C

import pytest
import torch

import sparse_moe_layer_05_amd as moe
from sparse_moe_layer_05_amd import binding as B

FAKE = C.c_void_p(0x10000)
BAD, UNS, WS, OK = B.MOE_ERR_INVALID_ARG, B.MOE_ERR_UNSUPPORTED, B.MOE_ERR_WORKSPACE, B.MOE_OK


def desc(**kw):
    d = B.MoeDesc()
    base = dict(T=4, H=256, E=16, k=2, I=128, I_shared=0, latent=0, act_dtype=1, expert_dtype=1,
                flags=0)
    base.update(kw)
    for n, v in base.items():
        setattr(d, n, v)
    return d


def size(d):
    n = C.c_size_t(0)
    return moe.lib().moe_few_workspace_size(C.byref(d), C.byref(n)), n.value


@pytest.mark.parametrize("kw,code", [
    (dict(), OK), (dict(T=16), OK), (dict(T=0), OK), (dict(T=17), UNS), (dict(T=-1), BAD),
    (dict(latent=64), OK), (dict(latent=40), BAD), (dict(k=17), BAD), (dict(E=1024, k=64), OK),
    (dict(act_dtype=0, expert_dtype=0), UNS), (dict(expert_dtype=B.MOE_FP8_E4M3), OK),
    (dict(expert_dtype=B.MOE_MXFP4), OK), (dict(expert_dtype=B.MOE_MXFP4, I=144), BAD),
    (dict(expert_dtype=B.MOE_MXFP8, T=16, H=4096), OK),
    (dict(expert_dtype=B.MOE_MXFP8, T=16, H=4128), UNS),     # T * D over 65536
    (dict(expert_dtype=B.MOE_MXFP8, T=16, H=8192, latent=1024), OK),
    (dict(expert_dtype=B.MOE_FP8_E4M3, T=16, I=4096), OK),
    (dict(expert_dtype=B.MOE_FP8_E4M3, T=16, I=4112), UNS),  # T * I over 65536
    (dict(T=16, H=8192), OK),                                # bf16: no such bound
    (dict(flags=B.PATH_STREAM), BAD), (dict(flags=B.PATH_GROUPED), BAD), (dict(flags=3), BAD),
    (dict(flags=B.SAVED_IN_WORKSPACE), BAD), (dict(flags=B.ROUTING_GIVEN), OK),
    (dict(expert_dtype=B.MOE_MXFP4, flags=B.MX_GROUPED), BAD),
])
def test_few_descriptors(kw, code):
    assert size(desc(**kw))[0] == code


def test_few_argument_errors_are_reported_before_launch():
    w = B.MoeWeights()
    for n, _ in B.MoeWeights._fields_:
        setattr(w, n, FAKE.value)

    def call(d, y=FAKE, ws=FAKE, ws_bytes=1 << 40, r=None):
        return moe.lib().moe_few_forward(C.byref(d), C.byref(w), y, ws, ws_bytes,
                                         C.byref(r) if r else None, None)

    assert call(desc(T=0)) == OK
    assert call(desc(T=17)) == UNS
    assert call(desc(), y=None) == BAD
    assert call(desc(), y=C.c_void_p(0x10008)) == BAD
    assert call(desc(), ws=None) == WS and call(desc(), ws_bytes=size(desc())[1] - 1) == WS
    assert call(desc(flags=B.ROUTING_GIVEN)) == BAD
    assert call(desc(flags=B.ROUTING_GIVEN), r=B.MoeRouting()) == BAD
    for name, d in (("W_up", desc()), ("W_r", desc()), ("Ws_up", desc(I_shared=64)),
                    ("W_out", desc(latent=64)), ("s_down", desc(expert_dtype=B.MOE_MXFP4))):
        keep = getattr(w, name)
        setattr(w, name, None)
        assert call(d) == BAD, name
        setattr(w, name, keep)
    n = C.c_size_t(0)
    assert moe.lib().moe_few_workspace_size(None, C.byref(n)) == BAD
    assert moe.lib().moe_few_workspace_size(C.byref(desc()), None) == BAD


def test_few_path_takes_its_own_workspace():
    bf = torch.bfloat16
    z = lambda *s: torch.zeros(*s, dtype=bf)  # noqa: E731
    with pytest.raises(ValueError):
        moe.Layer(z(2, 64), z(4, 64), torch.zeros(4), z(4, 32, 64), z(4, 64, 32), 2, path="few",
                  no_alloc=True)

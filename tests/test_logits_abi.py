"""The operators over logits at the C ABI without a GPU: argument errors are returned before
anything touches CUDA, and an empty batch launches nothing."""
import ctypes

import pytest

OK, INVALID, UNSUPPORTED = 0, 1, 2
FAKE = ctypes.c_void_p(0x100000)      # never dereferenced
FAR = ctypes.c_void_p(0x40000000)     # does not overlap FAKE's rows
ODD = ctypes.c_void_p(0x100001)
HALF = ctypes.c_void_p(0x100002)
BF16, F16, F32 = 0, 1, 2


@pytest.fixture(scope="module")
def lib():
    from deterministic_token_logprob_gb300 import build
    build.build()
    import deterministic_token_logprob_gb300 as rlk
    return rlk.lib()


def call(fn, defaults, **k):
    a = dict(defaults)
    assert set(k) <= set(a), k
    a.update(k)
    return fn(*a.values())


ROWS = dict(logits=FAKE, dtype=BF16, T=0, ld=4096, V_true=4096, temperature=1.0)
SCORE = dict(ROWS, y=FAKE, top_k=5, logp=FAKE, rank=FAKE, lse=FAKE, entropy=FAKE, top_ids=FAKE, top_logp=FAKE,
             err=None, stream=None)
OUT = dict(d=FAR, out_dtype=BF16, V=4096, out_ld=4096, err=None, stream=None)
TGRAD = dict(ROWS, y=FAKE, lse=FAKE, entropy=FAKE, g=FAKE, ge=FAKE, **OUT)
FWD = dict(ROWS, ids=FAKE, teacher=FAKE, K=5, loss=FAKE, lse=FAKE, err=None, stream=None)
BWD = dict(ROWS, ids=FAKE, teacher=FAKE, K=5, lse=FAKE, g=FAKE, **OUT)
BOTH = dict(ROWS, ids=FAKE, teacher=FAKE, K=5, g=FAKE, loss=FAKE, lse=FAKE, **OUT)


@pytest.mark.parametrize("name,args", [("rlk_token_logprobs", SCORE), ("rlk_token_logprobs_bwd", TGRAD),
                                       ("rlk_distill_topk_fwd", FWD), ("rlk_distill_topk_bwd", BWD),
                                       ("rlk_distill_topk_fwd_bwd", BOTH)])
def test_rows(lib, name, args):
    fn = getattr(lib, name)
    assert call(fn, args) == OK                                     # T = 0
    assert call(fn, args, logits=None) == OK
    assert call(fn, args, T=4, logits=None) == INVALID
    assert call(fn, args, T=4, logits=ODD) == INVALID
    assert call(fn, args, T=4, logits=HALF, dtype=F32) == INVALID
    assert call(fn, args, T=-1) == INVALID
    assert call(fn, args, dtype=3) == INVALID
    assert call(fn, args, dtype=-1) == INVALID
    assert call(fn, args, V_true=0) == INVALID
    assert call(fn, args, V_true=4097) == INVALID                   # beyond the row
    for tau in (0.0, -1.0, 1e-7, 1e7, float("nan"), float("inf")):
        assert call(fn, args, temperature=tau) == INVALID
    big = (1 << 20) + 1
    more = {"V": big, "out_ld": big} if "V" in args else {}
    assert call(fn, args, V_true=big, ld=big, **more) == UNSUPPORTED
    assert call(fn, args, T=(1 << 28) + 1) == UNSUPPORTED


def test_score_arguments(lib):
    f = lib.rlk_token_logprobs
    assert call(f, SCORE, T=4, top_k=-1) == INVALID
    assert call(f, SCORE, T=4, top_k=129) == UNSUPPORTED
    assert call(f, SCORE, T=4, y=None) == INVALID                   # logp and rank need targets
    assert call(f, SCORE, T=4, y=None, logp=None) == INVALID
    assert call(f, SCORE, T=4, top_ids=None) == INVALID
    assert call(f, SCORE, T=4, top_logp=None) == INVALID


@pytest.mark.parametrize("name,args", [("rlk_token_logprobs_bwd", TGRAD), ("rlk_distill_topk_bwd", BWD),
                                       ("rlk_distill_topk_fwd_bwd", BOTH)])
def test_gradient_arguments(lib, name, args):
    fn = getattr(lib, name)
    assert call(fn, args, V=4095) == INVALID                        # narrower than V_true
    assert call(fn, args, out_ld=4095) == INVALID
    assert call(fn, args, out_dtype=F16) == UNSUPPORTED             # bf16 logits
    assert call(fn, args, dtype=F32, out_dtype=F16) == UNSUPPORTED
    assert call(fn, args, dtype=F32, out_dtype=BF16) == OK
    assert call(fn, args, dtype=F32, out_dtype=F32) == OK
    assert call(fn, args, T=4, d=None) == INVALID
    assert call(fn, args, T=4, d=ctypes.c_void_p(0x40000001)) == INVALID
    assert call(fn, args, T=4, d=ctypes.c_void_p(0x100000 + 4096)) == INVALID             # overlaps the logits
    assert call(fn, args, T=4, d=FAKE, out_ld=8192) == INVALID                            # not the same rows
    assert call(fn, args, T=4, dtype=F32, logits=FAKE, d=FAKE, out_dtype=BF16) == INVALID  # not the same type
    assert call(fn, args, T=4, g=None) == INVALID


def test_token_gradient_arguments(lib):
    f = lib.rlk_token_logprobs_bwd
    assert call(f, TGRAD, T=4, y=None) == INVALID
    assert call(f, TGRAD, T=4, lse=None) == INVALID
    assert call(f, TGRAD, T=4, entropy=None) == INVALID             # g_entropy needs it


def test_distillation_arguments(lib):
    for name, args in (("rlk_distill_topk_fwd", FWD), ("rlk_distill_topk_bwd", BWD), ("rlk_distill_topk_fwd_bwd", BOTH)):
        fn = getattr(lib, name)
        assert call(fn, args, K=0) == INVALID
        assert call(fn, args, K=129) == UNSUPPORTED
        assert call(fn, args, T=4, ids=None) == INVALID
        assert call(fn, args, T=4, teacher=None) == INVALID
    assert call(lib.rlk_distill_topk_fwd, FWD, T=4, loss=None) == INVALID
    assert call(lib.rlk_distill_topk_fwd_bwd, BOTH, T=4, loss=None) == INVALID
    assert call(lib.rlk_distill_topk_bwd, BWD, T=4, lse=None) == INVALID

"""Which pairs of logits and gradient the operators over logits take at the C ABI: rows that share no byte,
though the arrays' envelopes meet (column slices of one wider buffer), and never rows that do. A call that is
taken reaches the launch, which fails without a GPU and is RLK_ERR_CUDA then; refusals come before that."""
import ctypes
import itertools

import pytest
import torch

INVALID, CUDA = 1, 4
BF16, F16, F32 = 0, 1, 2
SIZE = {BF16: 2, F16: 2, F32: 4}
BASE = 0x10000000                          # never dereferenced


@pytest.fixture(scope="module")
def lib():
    if torch.cuda.is_available():
        pytest.skip("the addresses are made up")
    from deterministic_token_logprob_gb300 import build
    build.build()
    import deterministic_token_logprob_gb300 as rlk
    return rlk.lib()


def calls(lib, dtype, T, ld, V_true, d, out_dtype, V, out_ld):
    p, q = ctypes.c_void_p(BASE), ctypes.c_void_p(0x7000000000)
    rows, out = (p, dtype, T, ld, V_true, 1.0), (ctypes.c_void_p(d), out_dtype, V, out_ld, None, None)
    return {lib.rlk_token_logprobs_bwd(*rows, q, q, q, q, q, *out),
            lib.rlk_distill_topk_bwd(*rows, q, q, 5, q, q, *out),
            lib.rlk_distill_topk_fwd_bwd(*rows, q, q, 5, q, q, q, *out)}


def refused(lib, *a):
    s = calls(lib, *a)
    assert s == {INVALID} or s == {CUDA}, s
    return s == {INVALID}


def test_slices_of_one_buffer(lib):
    # logits = buf[:, :V], dlogits = buf[:, V:2 V], and the other way round
    assert not refused(lib, BF16, 4, 2000, 1000, BASE + 2000, BF16, 1000, 2000)
    assert not refused(lib, F32, 4, 2000, 1000, BASE - 4000, F32, 1000, 2000)
    # fp32 logits with their bf16 gradient behind each row
    assert not refused(lib, F32, 4, 1500, 1000, BASE + 4000, BF16, 1000, 3000)
    # a column too many on either side
    assert refused(lib, BF16, 4, 2000, 1001, BASE + 2000, BF16, 1001, 2001)
    assert refused(lib, BF16, 4, 2000, 1001, BASE + 2000, BF16, 1001, 2000)
    assert refused(lib, BF16, 4, 2000, 1000, BASE + 2000, BF16, 1001, 2000)
    assert refused(lib, BF16, 4, 2000, 1000, BASE + 1998, BF16, 1000, 2000)


def test_against_the_bytes_themselves(lib):
    """Every placement of small rows: refused exactly where a byte is shared, or where the row distances
    differ and the envelopes meet."""
    for (dtype, out_dtype), T, ld, n, V, out_ld in itertools.product(
            ((BF16, BF16), (F32, F32), (F32, BF16)), (1, 2, 3), (8, 11), (3, 8), (8, 9), (9, 11, 16, 22)):
        if n > ld or V > out_ld or V < n:
            continue
        eb, ob = SIZE[dtype], SIZE[out_dtype]
        z = {BASE + t * ld * eb + i for t in range(T) for i in range(n * eb)}
        for off in range(-60 * ob, 60 * ob, ob):
            d = {BASE + off + t * out_ld * ob + i for t in range(T) for i in range(V * ob)}
            if off == 0 and dtype == out_dtype and (ld == out_ld or T == 1):
                continue                       # in place
            apart = max(z) < min(d) or max(d) < min(z)
            want = bool(z & d) if ld * eb == out_ld * ob or T == 1 else not apart
            assert refused(lib, dtype, T, ld, n, BASE + off, out_dtype, V, out_ld) == want, (dtype, out_dtype, T, ld, n, V, out_ld, off)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,out_dtype", [(torch.bfloat16, None), (torch.float16, None), (torch.float32, None),
                                             (torch.float32, torch.bfloat16)])
@pytest.mark.parametrize("T,V,n", [(5, 64, 61), (40, 5003, 5003), (700, 9001, 9000)])
def test_gradient_beside_the_logits(dtype, out_dtype, T, V, n):
    from deterministic_token_logprob_gb300 import build
    build.build()
    import deterministic_token_logprob_gb300 as rlk
    gen = torch.Generator(device="cuda").manual_seed(V)
    wide = torch.zeros((T, 2 * V + 8), dtype=dtype, device="cuda")
    z = wide[:, :V]
    z.copy_(torch.randn((T, V), generator=gen, device="cuda"))
    out = wide[:, V:2 * V] if out_dtype is None else wide.view(out_dtype)[:, 2 * V:3 * V]
    apart = z.clone()
    y = torch.randint(0, n, (T,), generator=gen, device="cuda")
    ids = torch.randint(0, n, (T, 7), generator=gen, device="cuda")
    t = torch.randn((T, 7), generator=gen, device="cuda")
    g = torch.rand(T, generator=gen, device="cuda")
    r = rlk.token_logprobs(apart, y, V_true=n)
    kw = dict(V_true=n, out_dtype=out_dtype)
    for call in (lambda x, **o: rlk.token_logprobs_bwd(x, y, r.lse, r.entropy, g, g, **kw, **o),
                 lambda x, **o: rlk.distill_topk_bwd(x, ids, t, r.lse, g, **kw, **o),
                 lambda x, **o: rlk.distill_topk_fwd_bwd(x, ids, t, g, **kw, **o)[2]):
        want = call(apart)
        assert torch.equal(call(z, out=out), want) and torch.equal(out, want)
        assert torch.equal(z, apart)

"""The operators around the head at the C ABI without a GPU: argument errors are returned before
anything touches CUDA, and an empty batch launches nothing."""
import array
import ctypes

import pytest

OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3
FAKE = ctypes.c_void_p(0x100000)      # never dereferenced
FAR = ctypes.c_void_p(0x4000000000)   # meets none of FAKE's rows
ODD = ctypes.c_void_p(0x100001)
HALF = ctypes.c_void_p(0x100002)
BF16, F16, F32 = 0, 1, 2
BIG = 1 << 50


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


LOOKUP = dict(table=FAKE, dtype=BF16, V=4096, H=64, ld=64, start=0, V_true=4096, ids=FAKE, T=0, scale=1.0, out=FAR,
              out_dtype=BF16, out_ld=64, err=None, stream=None)
TABLE = dict(dout=FAKE, dtype=BF16, T=300, H=64, ld=64, ids=FAKE, V=4096, start=0, V_true=4096, scale=1.0, dW=FAR, add=1,
             err=None, ws=None, ws_bytes=0, stream=None)
NORM = dict(x=FAKE, dtype=BF16, T=0, H=64, ld=64, w=FAKE, b=FAKE, wdtype=F32, centered=1, eps=1e-5, y=FAR, out_dtype=BF16,
            out_ld=64, mean=FAKE, rstd=FAKE, err=None, stream=None)
GRAD = dict(dy=FAKE, dy_dtype=BF16, dy_ld=64, x=FAKE, dtype=BF16, ld=64, T=4, H=64, w=FAKE, wdtype=F32, mean=FAKE,
            rstd=FAKE, dx=FAR, dx_ld=64, dw=FAKE, db=FAKE, err=None, ws=None, ws_bytes=0, stream=None)


def test_lookup_arguments(lib):
    f = lib.rlk_embedding_fwd
    assert call(f, LOOKUP) == OK
    assert call(f, LOOKUP, ids=None, out=None) == OK                # T = 0
    assert call(f, LOOKUP, T=4, ids=None) == INVALID
    assert call(f, LOOKUP, T=4, out=None) == INVALID
    assert call(f, LOOKUP, table=None) == INVALID
    assert call(f, LOOKUP, table=ODD) == INVALID
    assert call(f, LOOKUP, T=4, dtype=F32, out_dtype=F32, table=HALF) == INVALID
    assert call(f, LOOKUP, T=-1) == INVALID
    assert call(f, LOOKUP, dtype=3) == INVALID
    assert call(f, LOOKUP, out_dtype=-1) == INVALID
    assert call(f, LOOKUP, out_dtype=F32) == UNSUPPORTED
    assert call(f, LOOKUP, dtype=F32) == OK                         # fp32 -> bf16
    assert call(f, LOOKUP, H=0) == INVALID
    assert call(f, LOOKUP, ld=63) == INVALID
    assert call(f, LOOKUP, out_ld=63) == INVALID
    for k in ("V", "V_true"):
        assert call(f, LOOKUP, **{k: 0}) == INVALID
        assert call(f, LOOKUP, **{k: (1 << 24) + 1}) == UNSUPPORTED
    assert call(f, LOOKUP, start=-1) == INVALID
    assert call(f, LOOKUP, H=(1 << 16) + 1, ld=1 << 17, out_ld=1 << 17) == UNSUPPORTED
    assert call(f, LOOKUP, T=(1 << 24) + 1) == UNSUPPORTED
    for s in (float("nan"), float("inf"), 1e39):
        assert call(f, LOOKUP, scale=s) == INVALID
    assert call(f, LOOKUP, T=4, out=FAKE) == INVALID                # over the table
    assert call(f, LOOKUP, T=4, out=ctypes.c_void_p(0x100000 + 4096 * 128 - 2)) == INVALID


def test_table_gradient_arguments(lib):
    f = lib.rlk_embedding_bwd
    assert call(f, TABLE) == WORKSPACE
    need = lib.rlk_embedding_bwd_workspace(300, 64)
    assert call(f, TABLE, ws=FAKE, ws_bytes=need - 1) == WORKSPACE
    assert call(f, TABLE, ws=HALF, ws_bytes=need) == WORKSPACE
    assert call(f, TABLE, T=0) == OK                                # nothing to add
    assert call(f, TABLE, T=0, dW=None) == INVALID
    more = dict(ws=FAKE, ws_bytes=BIG)
    assert call(f, TABLE, ids=None, **more) == INVALID
    assert call(f, TABLE, dout=None, **more) == INVALID
    assert call(f, TABLE, dout=ODD, **more) == INVALID
    assert call(f, TABLE, dW=HALF, **more) == INVALID
    assert call(f, TABLE, dW=FAKE, **more) == INVALID               # over dout
    assert call(f, TABLE, ld=63, **more) == INVALID
    assert call(f, TABLE, dtype=3, **more) == INVALID
    assert call(f, TABLE, V=0, **more) == INVALID
    assert call(f, TABLE, start=-1, **more) == INVALID
    assert call(f, TABLE, V_true=0, **more) == INVALID
    assert call(f, TABLE, scale=float("nan"), **more) == INVALID
    assert call(f, TABLE, T=-1, **more) == INVALID
    assert call(f, TABLE, T=(1 << 24) + 1, **more) == UNSUPPORTED
    assert call(f, TABLE, V=(1 << 24) + 1, **more) == UNSUPPORTED
    assert call(f, TABLE, H=(1 << 16) + 1, ld=1 << 17, **more) == UNSUPPORTED
    assert lib.rlk_embedding_bwd_workspace(0, 64) == lib.rlk_embedding_bwd_workspace(256, 64) == 0
    assert lib.rlk_embedding_bwd_workspace(-1, 64) == 0


def test_norm_arguments(lib):
    f = lib.rlk_layer_norm_fwd
    assert call(f, NORM) == OK
    assert call(f, NORM, x=None, y=None, w=None, b=None, mean=None, rstd=None) == OK
    for k in ("x", "y"):
        assert call(f, NORM, T=4, **{k: None}) == INVALID
        assert call(f, NORM, T=4, **{k: ODD}) == INVALID
    assert call(f, NORM, T=-1) == INVALID
    assert call(f, NORM, H=0) == INVALID
    assert call(f, NORM, ld=63) == INVALID
    assert call(f, NORM, out_ld=63) == INVALID
    assert call(f, NORM, dtype=3) == INVALID
    assert call(f, NORM, out_dtype=F16) == UNSUPPORTED
    assert call(f, NORM, wdtype=3) == INVALID
    assert call(f, NORM, wdtype=F16) == INVALID                     # neither the rows' type nor fp32
    assert call(f, NORM, wdtype=F16, w=None, b=None) == OK
    assert call(f, NORM, wdtype=F32, w=HALF) == INVALID
    for eps in (0.0, -1.0, 1e-19, 2.0, float("nan"), float("inf")):
        assert call(f, NORM, eps=eps) == INVALID
    assert call(f, NORM, H=(1 << 16) + 1, ld=1 << 17, out_ld=1 << 17) == UNSUPPORTED
    assert call(f, NORM, T=(1 << 24) + 1) == UNSUPPORTED
    assert call(f, NORM, T=4, y=ctypes.c_void_p(0x100080)) == INVALID              # shifted rows
    assert call(f, NORM, T=4, dtype=F32, out_dtype=BF16, y=FAKE) == INVALID        # not the same type
    assert call(f, NORM, T=4, y=FAKE, out_ld=128) == INVALID                       # nor the same rows


def test_norm_gradient_arguments(lib):
    f = lib.rlk_layer_norm_bwd
    assert call(f, GRAD) == WORKSPACE
    need = lib.rlk_layer_norm_bwd_workspace(4, 64)
    assert call(f, GRAD, ws=FAKE, ws_bytes=need - 1) == WORKSPACE
    assert call(f, GRAD, ws=HALF, ws_bytes=need) == WORKSPACE
    more = dict(ws=FAKE, ws_bytes=BIG)
    for k in ("x", "dy", "rstd"):
        assert call(f, GRAD, **{k: None}, **more) == INVALID
    for k in ("x", "dy", "dx"):
        assert call(f, GRAD, **{k: ODD}, **more) == INVALID
    for k in ("ld", "dy_ld", "dx_ld"):
        assert call(f, GRAD, **{k: 63}, **more) == INVALID
    assert call(f, GRAD, dx=None, dw=None, db=None, **more) == INVALID
    assert call(f, GRAD, T=0, dw=None, db=None) == OK
    assert call(f, GRAD, dtype=F32, dy_dtype=F16, **more) == UNSUPPORTED
    assert call(f, GRAD, dy_dtype=F32, **more) == UNSUPPORTED
    assert call(f, GRAD, wdtype=F16, **more) == INVALID
    assert call(f, GRAD, T=-1, **more) == INVALID
    assert call(f, GRAD, T=(1 << 24) + 1, **more) == UNSUPPORTED
    assert call(f, GRAD, dx=ctypes.c_void_p(0x100080), **more) == INVALID          # shifted rows of x and dy
    assert call(f, GRAD, dx=FAKE, dx_ld=128, **more) == INVALID
    assert call(f, GRAD, dtype=F32, dy_dtype=BF16, x=FAR, dx=FAKE, **more) == INVALID   # dy is not of dx's type
    assert lib.rlk_layer_norm_bwd_workspace(0, 64) == 0


class Tensors:
    def __init__(self, lib, at=(0x100000, 0x200000), n=(100, 50), dtypes=(F32, BF16), to=None, odtypes=None):
        self.lib, self.k = lib, len(at)
        self.a = [array.array(c, v) for c, v in (("Q", at), ("q", n), ("i", dtypes), ("Q", at if to is None else to),
                                                 ("i", dtypes if odtypes is None else odtypes))]

    def address(self, i):
        return ctypes.c_void_p(self.a[i].buffer_info()[0])

    def norm(self, n=None, norm=FAKE, ws=None, ws_bytes=0, **null):
        a = [None if k in null else self.address(i) for i, k in enumerate(("grads", "sizes", "dtypes"))]
        return self.lib.rlk_grad_norm(*a, self.k if n is None else n, norm, None, ws, ws_bytes, None)

    def clip(self, max_norm=1.0, norm=FAR, ws=None, ws_bytes=0, **null):
        a = [None if k in null else self.address(i) for i, k in enumerate(("grads", "sizes", "dtypes", "outs", "odtypes"))]
        return self.lib.rlk_clip_grad_norm(*a[:3], self.k, max_norm, *a[3:], norm, None, ws, ws_bytes, None)


def test_gradient_norm_arguments(lib):
    t = Tensors(lib)
    need = lib.rlk_grad_norm_workspace(2)
    assert t.norm() == WORKSPACE
    assert t.norm(ws=FAKE, ws_bytes=need - 1) == WORKSPACE
    assert t.norm(ws=HALF, ws_bytes=need) == WORKSPACE
    assert t.norm(n=-1) == INVALID
    assert t.norm(n=(1 << 14) + 1) == UNSUPPORTED
    assert t.norm(norm=None) == INVALID
    for k in ("grads", "sizes", "dtypes"):
        assert t.norm(**{k: None}) == INVALID
    assert Tensors(lib, at=(0x100002, 0x200000)).norm() == INVALID          # misaligned
    assert Tensors(lib, at=(0, 0x200000)).norm() == INVALID
    assert Tensors(lib, at=(0, 0x200000), n=(0, 5)).norm() == WORKSPACE     # an empty tensor needs no address
    assert Tensors(lib, n=(-1, 5)).norm() == INVALID
    assert Tensors(lib, n=((1 << 40) + 1, 5)).norm() == UNSUPPORTED
    assert Tensors(lib, dtypes=(3, 0)).norm() == INVALID
    assert Tensors(lib, at=(0x100000, 0x100000)).norm() == WORKSPACE        # twice the same: it counts twice


def test_clip_arguments(lib):
    t = Tensors(lib)
    assert t.clip() == WORKSPACE                                            # in place
    for m in (0.0, -1.0, float("nan")):
        assert t.clip(max_norm=m) == INVALID
    assert t.clip(max_norm=float("inf")) == WORKSPACE
    assert t.clip(norm=None) == INVALID
    for k in ("outs", "odtypes"):
        assert t.clip(**{k: None}) == INVALID
    assert Tensors(lib, odtypes=(BF16, F32)).clip() == UNSUPPORTED          # bf16 -> fp32
    assert Tensors(lib, odtypes=(F16, BF16)).clip() == UNSUPPORTED
    assert Tensors(lib, odtypes=(3, BF16)).clip() == INVALID
    assert Tensors(lib, to=(0x300000, 0x400000), odtypes=(BF16, BF16)).clip() == WORKSPACE
    assert Tensors(lib, to=(0x100000, 0x400000), odtypes=(BF16, BF16)).clip() == INVALID   # over itself in another type
    assert Tensors(lib, to=(0x300000, 0)).clip() == INVALID
    assert Tensors(lib, to=(0x300000, 0x400001)).clip() == INVALID
    assert Tensors(lib, at=(0x100000, 0x100000)).clip() == INVALID          # twice the same: scaled twice
    assert Tensors(lib, to=(0x300000, 0x300000)).clip() == INVALID          # two results in one place
    assert Tensors(lib, to=(0x200010, 0x400000)).clip() == INVALID          # a result over another gradient
    assert Tensors(lib, to=(0x100004, 0x400000)).clip() == INVALID          # over its own, shifted
    assert Tensors(lib, at=(0x200000, 0x100000)).clip() == WORKSPACE        # any order of addresses
    # side by side
    assert Tensors(lib, at=(0x100000, 0x100000 + 400), n=(100, 50), dtypes=(F32, F32)).clip() == WORKSPACE
    assert Tensors(lib, at=(0x100000, 0x100000 + 396), n=(100, 50), dtypes=(F32, F32)).clip() == INVALID
    # the norm over a gradient or a result
    for norm in (0x100000, 0x100004, 0x200000):
        assert Tensors(lib).clip(norm=norm) == INVALID
        assert Tensors(lib).norm(norm=norm) == WORKSPACE
    assert Tensors(lib, to=(0x300000, 0x400000), odtypes=(BF16, BF16)).clip(norm=0x400000) == INVALID
    assert Tensors(lib, to=(0x300000, 0x400000), odtypes=(BF16, BF16)).clip(norm=0x500000) == WORKSPACE

"""Host-side checks of the embedding's, the norm's and the 8-bit checkpoint's
entry points: no GPU needed.

Every rejected call passes null data pointers or pointers that nothing reads
(the checks come first and nothing is enqueued); the binding refuses wrong
shapes, types and places before it calls the library."""

import ctypes
import os

import pytest
import torch

from uniform_noise_diffusion_amd import binding as B

NULL = None
FAKE = ctypes.c_void_p(4096)  # never read: another argument is refused
ODD = ctypes.c_void_p(4097)


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(B.LIB_PATH):
        pytest.skip("libmdlm.so not built")
    return B.load()


def call(fn, order, args, kw):
    a = dict(args, **kw)
    return fn(*[a[k] for k in order])


EMBED = ("ids", "n", "table", "dt", "V", "H", "scale", "out", "st")
GRAD = ("ids", "n", "g", "dt", "V", "H", "scale", "d", "acc", "ws", "wsb", "st")
FWD = ("x", "dt", "n", "H", "kind", "w", "b", "eps", "y", "mean", "rstd", "q", "qe", "st")
BWD = ("dy", "x", "dt", "n", "H", "kind", "w", "mean", "rstd", "dx", "dw", "db", "acc", "ws",
       "wsb", "st")
BWD8 = ("dy", "q", "qe", "dt", "n", "H", "kind", "w", "mean", "rstd", "dx", "dw", "db", "acc",
        "ws", "wsb", "st")


@pytest.mark.parametrize("kw,code,msg", [
    (dict(dt=3), B.MDLM_EINVAL, "dtype"),
    (dict(n=-1), B.MDLM_EINVAL, "bad sizes"),
    (dict(H=0), B.MDLM_EINVAL, "bad sizes"),
    (dict(n=1 << 31), B.MDLM_EUNSUPPORTED, "below 2^31"),
    (dict(H=(1 << 26) + 1), B.MDLM_EUNSUPPORTED, "exceeds 67108864"),
    (dict(H=(1 << 31) - 1), B.MDLM_EUNSUPPORTED, "exceeds 67108864"),
    (dict(V=0), B.MDLM_EINVAL, "V must"),
    (dict(scale=float("nan")), B.MDLM_EINVAL, "finite"),
    (dict(scale=float("inf")), B.MDLM_EINVAL, "finite"),
    (dict(), B.MDLM_EINVAL, "null pointer"),
    (dict(ids=FAKE, table=ODD, out=FAKE), B.MDLM_EINVAL, "aligned"),
])
def test_embed_refuses(lib, kw, code, msg):
    base = dict(ids=NULL, n=4, table=NULL, dt=1, V=8, H=64, scale=1.0, out=NULL, st=NULL)
    assert call(lib.mdlm_embed, EMBED, base, kw) == code
    assert msg in B.mdlm_last_error()


@pytest.mark.parametrize("kw,code,msg", [
    (dict(dt=-1), B.MDLM_EINVAL, "dtype"),
    (dict(n=-5), B.MDLM_EINVAL, "bad sizes"),
    (dict(n=1 << 31), B.MDLM_EUNSUPPORTED, "below 2^31"),
    (dict(H=(1 << 26) + 1), B.MDLM_EUNSUPPORTED, "exceeds 67108864"),
    (dict(n=0, H=(1 << 31) - 1), B.MDLM_EUNSUPPORTED, "exceeds 67108864"),
    (dict(V=-2), B.MDLM_EINVAL, "V must"),
    (dict(scale=float("-inf")), B.MDLM_EINVAL, "finite"),
    (dict(acc=2), B.MDLM_EINVAL, "accumulate"),
    (dict(), B.MDLM_EINVAL, "null pointer"),
    (dict(n=0), B.MDLM_EINVAL, "null pointer"),
    (dict(ids=FAKE, g=FAKE, d=ODD), B.MDLM_EINVAL, "aligned"),
    (dict(ids=FAKE, g=FAKE, d=FAKE), B.MDLM_EWORKSPACE, "workspace of 0 bytes"),
    (dict(ids=FAKE, g=FAKE, d=FAKE, ws=FAKE, wsb=16), B.MDLM_EWORKSPACE, "need"),
    (dict(ids=FAKE, g=FAKE, d=FAKE, ws=ctypes.c_void_p(4096 + 16), wsb=1 << 30), B.MDLM_EINVAL,
     "256-byte"),
])
def test_embed_grad_refuses(lib, kw, code, msg):
    base = dict(ids=NULL, n=4000, g=NULL, dt=1, V=8, H=64, scale=1.0, d=NULL, acc=0, ws=NULL,
                wsb=0, st=NULL)
    assert call(lib.mdlm_embed_grad, GRAD, base, kw) == code
    assert msg in B.mdlm_last_error()


@pytest.mark.parametrize("kw,code,msg", [
    (dict(dt=9), B.MDLM_EINVAL, "dtype"),
    (dict(n=-1), B.MDLM_EINVAL, "bad sizes"),
    (dict(H=16385), B.MDLM_EUNSUPPORTED, "exceeds 16384"),
    (dict(kind=2), B.MDLM_EINVAL, "unknown norm"),
    (dict(eps=0.0), B.MDLM_EINVAL, "eps"),
    (dict(eps=-1.0), B.MDLM_EINVAL, "eps"),
    (dict(eps=float("nan")), B.MDLM_EINVAL, "eps"),
    (dict(eps=1e-60), B.MDLM_EINVAL, "eps"),
    (dict(eps=1e60), B.MDLM_EINVAL, "eps"),
    (dict(), B.MDLM_EINVAL, "null pointer"),
    (dict(x=FAKE, y=FAKE, q=FAKE), B.MDLM_EINVAL, "together"),
    (dict(x=FAKE, y=FAKE, qe=FAKE), B.MDLM_EINVAL, "together"),
    (dict(x=FAKE, y=ODD), B.MDLM_EINVAL, "aligned"),
    (dict(x=FAKE, y=FAKE, rstd=ctypes.c_void_p(4098)), B.MDLM_EINVAL, "aligned"),
])
def test_norm_fwd_refuses(lib, kw, code, msg):
    base = dict(x=NULL, dt=1, n=4, H=64, kind=0, w=NULL, b=NULL, eps=1e-5, y=NULL, mean=NULL,
                rstd=NULL, q=NULL, qe=NULL, st=NULL)
    assert call(lib.mdlm_norm_fwd, FWD, base, kw) == code
    assert msg in B.mdlm_last_error()


IN = dict(dy=FAKE, x=FAKE, q=FAKE, qe=FAKE, mean=FAKE, rstd=FAKE)


@pytest.mark.parametrize("entry", ["mdlm_norm_bwd", "mdlm_norm_bwd_ckpt8"])
@pytest.mark.parametrize("kw,code,msg", [
    (dict(dt=2), B.MDLM_EINVAL, "dtype"),
    (dict(H=0), B.MDLM_EINVAL, "bad sizes"),
    (dict(H=1 << 20), B.MDLM_EUNSUPPORTED, "exceeds"),
    (dict(kind=-1), B.MDLM_EINVAL, "unknown norm"),
    (dict(acc=-1), B.MDLM_EINVAL, "accumulate"),
    (dict(dx=FAKE), B.MDLM_EINVAL, "null input"),
    (dict(IN, dx=FAKE, mean=NULL), B.MDLM_EINVAL, "null input"),
    (dict(IN, dx=FAKE, rstd=NULL), B.MDLM_EINVAL, "null input"),
    (dict(IN, dx=FAKE, x=NULL, q=NULL), B.MDLM_EINVAL, "null input"),
    (IN, B.MDLM_EINVAL, "no gradient"),
    (dict(IN, dx=ODD), B.MDLM_EINVAL, "aligned"),
    (dict(IN, dw=FAKE), B.MDLM_EWORKSPACE, "workspace of 0"),
    (dict(IN, db=FAKE, ws=FAKE, wsb=8), B.MDLM_EWORKSPACE, "need"),
    (dict(IN, db=FAKE, ws=ctypes.c_void_p(4100), wsb=1 << 20), B.MDLM_EINVAL, "256-byte"),
])
def test_norm_bwd_refuses(lib, entry, kw, code, msg):
    base = dict(dy=NULL, x=NULL, q=NULL, qe=NULL, dt=1, n=4, H=64, kind=0, w=NULL, mean=NULL,
                rstd=NULL, dx=NULL, dw=NULL, db=NULL, acc=0, ws=NULL, wsb=0, st=NULL)
    order = BWD if entry == "mdlm_norm_bwd" else BWD8
    assert call(getattr(lib, entry), order, base, kw) == code
    assert msg in B.mdlm_last_error()


def test_ckpt8_refuses(lib):
    for args, code, msg in [
            ((NULL, 7, 4, 64, NULL, NULL, NULL), B.MDLM_EINVAL, "dtype"),
            ((NULL, 1, -4, 64, NULL, NULL, NULL), B.MDLM_EINVAL, "bad sizes"),
            ((NULL, 1, 4, 0, NULL, NULL, NULL), B.MDLM_EINVAL, "bad sizes"),
            ((NULL, 1, (1 << 31) - 1, 1 << 20, NULL, NULL, NULL), B.MDLM_EUNSUPPORTED, "blocks"),
            ((FAKE, 1, 4, 64, FAKE, NULL, NULL), B.MDLM_EINVAL, "null pointer"),
            ((ODD, 1, 4, 64, FAKE, FAKE, NULL), B.MDLM_EINVAL, "aligned")]:
        assert lib.mdlm_ckpt8_save(*args) == code
        assert msg in B.mdlm_last_error()
        x, dt, n, H, q, qe, st = args
        assert lib.mdlm_ckpt8_load(q, qe, dt, n, H, x, st) == code
        assert msg in B.mdlm_last_error()


def test_check_tokens_refuses(lib):
    assert lib.mdlm_check_tokens(NULL, -1, 8, FAKE, NULL) == B.MDLM_EINVAL
    assert lib.mdlm_check_tokens(NULL, 4, 0, FAKE, NULL) == B.MDLM_EINVAL
    assert lib.mdlm_check_tokens(NULL, 4, 8, FAKE, NULL) == B.MDLM_EINVAL
    assert lib.mdlm_check_tokens(FAKE, 4, 8, NULL, NULL) == B.MDLM_EINVAL


def test_workspace_sizes(lib):
    assert B.mdlm_embed_grad_workspace_bytes(0, 64) == 0
    assert B.mdlm_embed_grad_workspace_bytes(-1, 64) == 0
    assert B.mdlm_embed_grad_workspace_bytes(5, 0) == 0
    assert B.mdlm_embed_grad_workspace_bytes(1 << 31, 64) == 0
    assert B.mdlm_embed_grad_workspace_bytes(1024, 100) == 0  # few tokens need none
    sizes = [B.mdlm_embed_grad_workspace_bytes(n, 100) for n in (1025, 1500, 5000, 1 << 20)]
    assert all(s > 0 for s in sizes) and sizes == sorted(sizes)
    assert B.mdlm_norm_bwd_workspace_bytes(0, 64) == 0
    assert B.mdlm_norm_bwd_workspace_bytes(4, 16385) == 0
    assert B.mdlm_norm_bwd_workspace_bytes(4, -1) == 0
    assert B.mdlm_norm_bwd_workspace_bytes(1, 64) > 0


# ---- the binding's own refusals (CPU tensors: nothing can reach the library) --


def _bf(*shape):
    return torch.zeros(shape, dtype=torch.bfloat16)


def test_binding_refuses_host_tensors():
    ids = torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError, match="device"):
        B.mdlm_embed(ids, _bf(8, 16), 1.0, _bf(3, 16))
    with pytest.raises(ValueError, match="device"):
        B.mdlm_embed_grad(ids, _bf(3, 16), 1.0, torch.zeros(8, 16))
    with pytest.raises(ValueError, match="device"):
        B.mdlm_norm_fwd(_bf(3, 16), 0, None, None, 1e-5, _bf(3, 16))
    with pytest.raises(ValueError, match="device"):
        B.mdlm_norm_bwd(_bf(3, 16), _bf(3, 16), 1, None, None, torch.zeros(3), _bf(3, 16))
    with pytest.raises(ValueError, match="device"):
        B.mdlm_ckpt8_save(_bf(3, 16), torch.zeros(3, 16, dtype=torch.uint8),
                          torch.zeros(3, 1, dtype=torch.uint8))


def test_binding_refuses_wrong_types_and_shapes():
    ids = torch.zeros(3, dtype=torch.int32, device="meta")

    def m(*shape, dtype=torch.bfloat16):
        return torch.zeros(shape, dtype=dtype, device="meta")

    with pytest.raises(ValueError, match=r"\[V, H\]"):
        B.mdlm_embed(ids, m(16), 1.0, m(3, 16))
    with pytest.raises(ValueError, match="device tensor"):
        B.mdlm_embed(ids, m(8, 16), 1.0, m(3, 16))
    with pytest.raises(TypeError, match="float32"):
        B._arg(m(8, 16), "d_table", torch.float32, (8, 16), -1)
    with pytest.raises(ValueError, match="shape"):
        B._ckpt8_args(m(3, 130, dtype=torch.uint8), m(3, 1, dtype=torch.uint8), (3, 130), -1)
    with pytest.raises(TypeError, match="unsupported element type"):
        B.dtype_code(m(2, dtype=torch.float16))


def test_launch_makes_the_tensors_device_current(monkeypatch):
    """The library launches on the current device: a call on another device's
    tensors switches to it, and back."""
    seen, now = [], [0]

    class Device:
        def __init__(self, index):
            self.index = index

        def __enter__(self):
            self.was, now[0] = now[0], self.index

        def __exit__(self, *exc):
            now[0] = self.was

    monkeypatch.setattr(torch.cuda, "current_device", lambda: now[0])
    monkeypatch.setattr(torch.cuda, "device", Device)
    monkeypatch.setattr(B, "_raw_stream", lambda dev: 1000 + dev)

    def fn(*args):
        seen.append((now[0], args))
        return B.MDLM_OK

    B._launch(fn, 0, None, "a")
    B._launch(fn, 3, None, "b")
    assert seen == [(0, ("a", 1000)), (3, ("b", 1003))] and now[0] == 0

    class Stream:
        device = torch.device("cuda", 2)
        cuda_stream = 77

    B._launch(fn, 2, Stream, "c")
    assert seen[-1] == (2, ("c", 77))
    with pytest.raises(ValueError, match="stream"):
        B._launch(fn, 1, Stream, "d")
    assert len(seen) == 3

"""Sizes past what the library's 32-bit arguments hold: refused by the binding
and by the library, no GPU needed.  The tensors are meta or expanded ones (they
take no memory), and the library replaced by one that must not be called."""

import ctypes
import os

import pytest
import torch

from uniform_noise_diffusion_amd import binding as B

PAST = (1 << 32) + 64  # what 32 bits keep of it is 64


@pytest.fixture
def no_library(monkeypatch):
    class Library:
        def __getattr__(self, name):
            raise AssertionError(f"{name} was reached")

    monkeypatch.setattr(B, "load", Library)


def meta(*shape, dtype=torch.bfloat16):
    return torch.empty(shape, dtype=dtype, device="meta")


def test_rows_past_int32(no_library):
    """One row of 2^32 + 64 entries must not go for one of 64."""
    for lead in ((), (1,)):
        x = meta(*lead, PAST)
        q = meta(*lead, PAST, dtype=torch.uint8)
        q_exp = meta(*lead, PAST // 128 + 1, dtype=torch.uint8)
        stat = meta(*lead, dtype=torch.float32)
        for call in (lambda: B.mdlm_ckpt8_save(x, q, q_exp),
                     lambda: B.mdlm_ckpt8_load(q, q_exp, x),
                     lambda: B.mdlm_norm_fwd(x, 1, None, None, 1e-5, x),
                     lambda: B.mdlm_norm_bwd(x, x, 1, None, None, stat, x),
                     lambda: B.mdlm_norm_bwd_ckpt8(x, q, q_exp, 1, None, None, stat, x)):
            with pytest.raises(ValueError, match="32 bits"):
                call()


@pytest.mark.parametrize("shape", [(PAST, 8), (8, PAST), (1 << 31, 8), (8, 1 << 31)])
def test_tables_past_int32(no_library, shape):
    ids = meta(3, dtype=torch.int32)
    table, rows = meta(*shape), meta(3, shape[1])
    with pytest.raises(ValueError, match="32 bits"):
        B.mdlm_embed(ids, table, 1.0, rows)
    with pytest.raises(ValueError, match="32 bits"):
        B.mdlm_embed_grad(ids, rows, 1.0, meta(*shape, dtype=torch.float32))


@pytest.mark.parametrize("name", [n for n in B.EXPORTED if n not in
                                  ("mdlm_set_checking", "mdlm_last_error", "mdlm_version")])
def test_numbers_past_int32(name):
    """No call takes the low 32 bits of a larger number for the number.  (The
    arguments are converted before the library is entered.)"""
    if not os.path.exists(B.LIB_PATH):
        pytest.skip("libmdlm.so not built")
    fn = getattr(B.load(), name)
    assert ctypes.c_int32 not in fn.argtypes
    args = [None if t is ctypes.c_void_p else 0 for t in fn.argtypes]
    for i in (i for i, t in enumerate(fn.argtypes) if t is B._Int32):
        for value in (PAST, 1 << 31, -(1 << 31) - 1):
            with pytest.raises(ctypes.ArgumentError, match="32 bits"):
                fn(*args[:i], value, *args[i + 1:])


@pytest.mark.parametrize("H,code", [((1 << 31) - 1, B.MDLM_EUNSUPPORTED),
                                    ((1 << 31) - 127, B.MDLM_EUNSUPPORTED),
                                    ((1 << 31) - 128, B.MDLM_OK)])
def test_checkpoint_rows_whose_last_block_ends_past_int32(H, code):
    """Columns are counted in 32 bits up to the end of a row's last block of
    128.  (Without rows nothing is launched.)"""
    if not os.path.exists(B.LIB_PATH):
        pytest.skip("libmdlm.so not built")
    lib = B.load()
    for dtype in (B.MDLM_BF16, B.MDLM_F32):
        assert lib.mdlm_ckpt8_save(None, dtype, 0, H, None, None, None) == code
        assert lib.mdlm_ckpt8_load(None, None, dtype, 0, H, None, None) == code
    if code != B.MDLM_OK:
        assert "exceeds 2147483520" in B.mdlm_last_error()

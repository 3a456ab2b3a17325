"""Refusals of the 4-bit and embedding calls, on the CPU: every check of an
argument comes before the first use of the GPU, so a refused call launches
nothing and needs no device.  The device addresses are made up and never read."""
from __future__ import annotations

import ctypes

import numpy as np
import pytest
import torch

import lossless_entropy_coded_canonical_b200 as dfw
from lossless_entropy_coded_canonical_b200 import LanesInfo, LanesScope, Q4Info, Table

A = 1 << 20  # an aligned device address (never dereferenced)


def q4_info(rows=16, cols=128, group=128, zeros=0):
    info = Q4Info(rows, cols, group, zeros, 0)
    assert dfw.lib().dfw_q4_query(ctypes.byref(info)) == dfw.OK
    return info


@pytest.mark.parametrize("rows,cols,group,zeros,tile,tiles", [
    (1, 32, 32, 0, 1024 + 128, 1), (16, 128, 128, 0, 1024 + 32, 1), (17, 128, 128, 1, 1024 + 48, 2),
    (16, 192, 64, 0, 1024 + 64, 2), (33, 4096, 32, 1, 1024 + 192, 3 * 32), (1 << 30, 65536, 128, 0, 1056, (1 << 26) * 512)])
def test_q4_query_bytes(rows, cols, group, zeros, tile, tiles):
    assert q4_info(rows, cols, group, zeros).bytes == tile * tiles


@pytest.mark.parametrize("rows,cols,group,zeros", [
    (0, 128, 128, 0), (16, 0, 32, 0), (16, 128, 16, 0), (16, 128, 96, 0), (16, 160, 64, 0), (16, 128, 128, 2),
    ((1 << 30) + 1, 128, 128, 0), (16, 65536 + 128, 128, 0)])
def test_q4_query_refuses(rows, cols, group, zeros):
    assert dfw.lib().dfw_q4_query(ctypes.byref(Q4Info(rows, cols, group, zeros, 0))) == dfw.EINVAL


def test_q4_query_refuses_null():
    assert dfw.lib().dfw_q4_query(None) == dfw.EINVAL


def test_q4_pack_and_quantise_refuse():
    lib, info, zinfo = dfw.lib(), q4_info(), q4_info(zeros=1)
    R, Z = ctypes.byref(info), ctypes.byref(zinfo)
    assert lib.dfw_q4_pack(A, A, None, None, A, None) == dfw.EINVAL
    assert lib.dfw_q4_pack(None, A, None, R, A, None) == dfw.EINVAL
    assert lib.dfw_q4_pack(A, None, None, R, A, None) == dfw.EINVAL
    assert lib.dfw_q4_pack(A, A, None, R, None, None) == dfw.EINVAL
    assert lib.dfw_q4_pack(A, A, A, R, A, None) == dfw.EINVAL      # zero points for a matrix without
    assert lib.dfw_q4_pack(A, A, None, Z, A, None) == dfw.EINVAL   # none for a matrix with
    assert lib.dfw_q4_pack(A + 2, A, None, R, A, None) == dfw.EALIGN
    assert lib.dfw_q4_pack(A, A + 1, None, R, A, None) == dfw.EALIGN
    assert lib.dfw_q4_pack(A, A, None, R, A + 8, None) == dfw.EALIGN
    assert lib.dfw_q4_quantise(None, 128, R, A, None) == dfw.EINVAL
    assert lib.dfw_q4_quantise(A, 127, R, A, None) == dfw.EINVAL
    assert lib.dfw_q4_quantise(A + 1, 128, R, A, None) == dfw.EALIGN
    assert lib.dfw_q4_dequantise(A, R, None, None) == dfw.EINVAL
    assert lib.dfw_q4_dequantise(A, R, A + 8, None) == dfw.EALIGN
    info.bytes += 16
    assert lib.dfw_q4_dequantise(A, R, A, None) == dfw.EINVAL


def test_q4_gemv_refuses():
    lib, info = dfw.lib(), q4_info(rows=48, cols=256)
    R = ctypes.byref(info)

    def call(packed=A, ref=R, m=2, x=A, ldx=256, y=A, fp32=1, ldy=48):
        return lib.dfw_q4_gemv(packed, ref, m, x, ldx, y, fp32, ldy, None)

    assert call(packed=None) == call(ref=None) == call(x=None) == call(y=None) == dfw.EINVAL
    assert call(m=65) == call(ldx=255) == call(ldy=47) == call(fp32=2) == dfw.EINVAL
    assert call(packed=A + 4) == call(x=A + 1) == call(y=A + 2) == call(y=A + 1, fp32=0) == dfw.EALIGN
    assert call(m=0) == dfw.OK  # nothing to do, no GPU needed
    info.bytes -= 16
    assert call() == dfw.EINVAL


def coded_scope(n=5000):
    u = (np.random.default_rng(0).standard_normal(n) * 0.02).astype(np.float32)
    enc = dfw.encode(torch.from_numpy(u).to(torch.bfloat16))
    pl = dfw.plan_lanes(enc)
    scope = LanesScope(A, A, A, A, A, ctypes.pointer(enc.table), ctypes.pointer(pl.info))
    return scope, enc, pl


def test_embed_lanes_refuses():
    lib = dfw.lib()
    scope, enc, pl = coded_scope()

    def call(s=scope, first=0, rows=50, dim=100, ids=A, wide=1, tokens=3, out=A, ld=100):
        return lib.dfw_embed_lanes(None if s is None else ctypes.byref(s), first, rows, dim, ids, wide, tokens, 1.0, out, ld,
                                   None)

    assert call(s=None) == call(ids=None) == call(out=None) == call(wide=2) == dfw.EINVAL
    assert call(rows=0) == call(dim=0) == call(rows=51) == call(first=1) == call(ld=99) == dfw.EINVAL
    assert call(first=5001, rows=1, dim=1) == call(rows=1 << 40) == call(dim=(1 << 20) + 1) == dfw.EINVAL
    assert call(tokens=(1 << 20) + 1) == dfw.EINVAL
    assert call(ids=A + 4) == call(ids=A + 2, wide=0) == call(out=A + 1) == dfw.EALIGN
    for field in ("d_stream", "d_mant", "d_lut", "d_chunk_bits", "d_group_start"):
        for value, want in ((None, dfw.EINVAL), (A + 8, dfw.EALIGN)):
            s = LanesScope(A, A, A, A, A, scope.table, scope.info)
            setattr(s, field, value)
            assert call(s=s) == want, field
    bad = Table.from_buffer_copy(enc.table)
    bad.len[120] = 40  # not a code
    assert call(s=LanesScope(A, A, A, A, A, ctypes.pointer(bad), scope.info)) == dfw.EINVAL
    info = LanesInfo.from_buffer_copy(pl.info)
    info.n_groups += 1
    assert call(s=LanesScope(A, A, A, A, A, scope.table, ctypes.pointer(info))) == dfw.EINVAL
    assert call(tokens=0, ids=None, out=None) == dfw.OK


def test_embed_rows_refuses():
    lib = dfw.lib()

    def call(table=A, rows=10, dim=64, ldt=64, ids=A, wide=0, tokens=2, out=A, ld=64):
        return lib.dfw_embed_rows(table, rows, dim, ldt, ids, wide, tokens, 1.0, out, ld, None)

    assert call(table=None) == call(ids=None) == call(out=None) == call(wide=-1) == dfw.EINVAL
    assert call(rows=0) == call(rows=(1 << 30) + 1) == call(dim=0) == call(ldt=63) == call(ld=63) == dfw.EINVAL
    assert call(tokens=(1 << 20) + 1) == dfw.EINVAL
    assert call(table=A + 1) == call(out=A + 1) == call(ids=A + 2) == call(ids=A + 4, wide=1) == dfw.EALIGN
    assert call(tokens=0, ids=None, out=None) == dfw.OK


def test_embed_grad_refuses():
    lib = dfw.lib()
    need = dfw.embed_grad_scratch_bytes(200, 64)
    assert need > 0 and dfw.embed_grad_scratch_bytes(7, 64) == 0  # few tokens need none

    def call(ids=A, wide=1, tokens=200, dy=A, dyf=1, ld=64, rows=9, dim=64, grad=A, gf=1, acc=0, scratch=A, nbytes=need):
        return lib.dfw_embed_grad(ids, wide, tokens, dy, dyf, ld, rows, dim, 1.0, grad, gf, acc, scratch, nbytes, None)

    assert call(ids=None) == call(dy=None) == call(grad=None) == call(scratch=None) == dfw.EINVAL
    assert call(wide=2) == call(dyf=2) == call(gf=-1) == call(acc=2) == call(ld=63) == dfw.EINVAL
    assert call(rows=0) == call(rows=(1 << 30) + 1) == call(dim=0) == call(dim=(1 << 20) + 1) == dfw.EINVAL
    assert call(tokens=(1 << 20) + 1) == dfw.EINVAL
    assert call(ids=A + 4) == call(dy=A + 2) == call(dy=A + 1, dyf=0) == call(grad=A + 2) == call(scratch=A + 8) == dfw.EALIGN
    assert call(nbytes=need - 1) == dfw.ENOMEM
    assert call(tokens=0, acc=1, ids=None, dy=None, scratch=None, nbytes=0) == dfw.OK


def test_binding_refuses_host_tensors_and_types():
    w = torch.zeros(16, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        dfw.q4_quantise(w)
    with pytest.raises(ValueError):
        dfw.q4_pack(torch.zeros(16, 64, dtype=torch.uint8), torch.zeros(16, 1, dtype=torch.bfloat16))
    with pytest.raises(ValueError):
        dfw.embed_rows(w, torch.zeros(3, dtype=torch.int64))
    with pytest.raises(ValueError):
        dfw.embed_grad(torch.zeros(3, dtype=torch.int64), torch.zeros(3, 8), 5)


def test_packed_weights_must_be_what_their_info_says():
    info = q4_info(33, 256, 64, 1)
    whole = torch.zeros(info.bytes + 16, dtype=torch.uint8)
    assert dfw.Q4Weights(whole[:info.bytes], info).shape == (33, 256)
    for packed in (whole, whole[:info.bytes - 1], whole[:info.bytes].view(torch.int8), torch.zeros(info.bytes * 2, dtype=torch.uint8)[::2]):
        with pytest.raises(ValueError):
            dfw.Q4Weights(packed, info)


def test_binding_refuses_packed_weights_on_the_host():
    """Packed weights may lie on the host (read from a file, say): not for these calls."""
    info = q4_info(16, 128, 128)
    q = dfw.Q4Weights(torch.zeros(info.bytes, dtype=torch.uint8), info)
    for call in (lambda: dfw.q4_dequantise(q), lambda: dfw.q4_gemv(q, torch.zeros(1, 128, dtype=torch.bfloat16))):
        with pytest.raises(ValueError, match="must be on a CUDA device"):
            call()

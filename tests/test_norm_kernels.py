"""Every compiled kernel of the norm is one that some call reaches: the rule that picks a kernel
(csrc/norm.cu), written out here over all widths and types, against the names in the built library."""
import re
import shutil
import subprocess

import pytest

from selective_state_space_32_b200 import build as B

BYTES = {"float": 4, "unsigned short": 2}
RING, BWD_THREADS, MAX_THREADS = 220 << 10, 640, 1024
WIDEST = 40000   # past it every width takes the same kernels


def up(a, b):
    return -(-a // b)


def row_shape(D, es):
    """(values of a vector, vectors a thread, threads a row, shifted); 0 vectors: several passes"""
    ve, shift = 16 // es, D * es % 16 != 0
    if shift and D <= 256:
        return 1, 8, 32, False
    n = up(D + ve - 1, ve) if shift else D // ve
    if not shift:
        for most, nv, threads in ((8, 1, 8), (16, 1, 16), (32, 1, 32), (64, 2, 32), (128, 4, 32)):
            if n <= most:
                return ve, nv, threads, False
        if es == 4 and n <= 256:
            return ve, 8, 32, False
    for most, nv in ((256, 1), (1024, 2), (4 * MAX_THREADS, 4)):
        if n <= most:
            return ve, nv, up(n, 32 * nv) * 32, shift
    return 1 if shift else ve, 0, 0, False


def bwd_smem(width, io, r, dres, stages):
    row = width * (BYTES[io] + (2 if dres else 1) * BYTES[r])
    return up(width * 4, 16) * 16 + stages * row


def forward_kernels():
    out = set()
    for io, r, res in (("float", "float", 0), ("float", "float", 1), ("unsigned short", "unsigned short", 0),
                       ("unsigned short", "unsigned short", 1), ("unsigned short", "float", 1)):
        for D in range(1, WIDEST):
            ve, nv, threads, shift = row_shape(D, BYTES[io])
            if nv == 0:
                out.add(("forward_long", io, r, res, ve))
            else:
                out.add(("forward", io, r, res, ve, nv, threads if threads <= 32 else 0, int(shift)))
    return out


def backward_kernels():
    out = set()
    for io, r in (("float", "float"), ("unsigned short", "unsigned short"), ("unsigned short", "float")):
        for dres in (False, True):
            for D in range(1, WIDEST):
                ve, nv, threads, shift = row_shape(D, BYTES[io])
                if nv and ve > 1:
                    n = up(D + ve - 1, ve) if shift else D // ve
                    two, most = bwd_smem(n * ve, io, r, dres, 2), 16 // ve
                    if bwd_smem(n * ve, io, r, dres, 1) > RING or n > most * BWD_THREADS:
                        ve, nv = 1 if shift else ve, 0
                    elif not (threads <= 32 and nv <= most):
                        want = BWD_THREADS // (1 if two * 2 > RING else 2 if two * 4 > RING else 4)
                        nv = 1
                        while nv < most and n > want * nv:
                            nv *= 2
                        threads = up(n, 32 * nv) * 32
                if nv == 0:
                    out.add(("backward_long", io, r, ve))
                elif threads <= 32:
                    out.add(("backward", io, r, ve, nv, threads, 4, 0))
                else:
                    out.add(("backward", io, r, ve, nv, 0, 1 if two > RING else 2, int(shift)))
    return out


def compiled():
    names = subprocess.run(["nm", "-C", B.build()], capture_output=True, text=True, check=True).stdout
    out = set()
    for kind, args in re.findall(r"norm_(\w+)_kernel<([^>]*)>\(sscan::norm::\wwdParams", names):
        vals = [{"true": "1", "false": "0"}.get(a.strip(), a.strip()) for a in args.split(",")]
        out.add((kind, *(int(v) if v.isdigit() else v for v in vals)))
    return out


@pytest.mark.skipif(shutil.which("nm") is None, reason="no nm")
def test_the_library_holds_the_kernels_that_calls_reach():
    have, want = compiled(), forward_kernels() | backward_kernels()
    assert have == want, (sorted(map(str, have - want)), sorted(map(str, want - have)))


def test_the_workspace_is_what_the_blocks_use():
    """Two rows of D sums a block: 148 blocks where every type takes several passes over a row, else at most 592."""
    from selective_state_space_32_b200 import sscan as S
    B.build()
    ws = S.lib().sscan_norm_backward_workspace_bytes
    for D in (10241, 10248, 12288, WIDEST):
        assert ws(3000, D) == up(2 * 148 * D * 4, 256) * 256
        assert ws(5, D) == up(2 * 5 * D * 4, 256) * 256
    for D in (64, 777, 5120, 10240):
        assert ws(3000, D) == up(2 * 592 * D * 4, 256) * 256

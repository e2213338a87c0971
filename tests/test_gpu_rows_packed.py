"""Rows of up to 4096 that share a wave, whatever their length, and calls of more rows than one
launch has threads for.

Codes and scales are the oracle's fp32 decision bit for bit; the last rows of a long call have the
bits of a call on those rows alone."""
import numpy as np
import pytest
import torch

import hadamard_rotated_precision_halo_amd as H
import oracle as O
import synth
from parity_util import (COUNTER64, CTR, DEV, KEY, Q_TORCH, SEED64, codes_to_np, signs_dev, to_dev)

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16

CASES = [
    # io, block, rows, cols, code type, signs, stochastic
    ("bf16", 64, 1, 192, O.I8, False, False),        # one row of a wave's 21
    ("bf16", 64, 85, 192, O.I8, True, True),         # four whole waves and one row
    ("bf16", 8, 64, 192, O.E4M3, True, False),       # blocks below a lane's 64 values
    ("f32", 64, 43, 320, O.E5M2, True, False),       # 12 rows a wave, 4 lanes idle
    ("bf16", 128, 42, 384, O.I8, False, True),       # 10 rows a wave
    ("bf16", 32, 30, 400, O.I8, False, False),       # padded to 416: the older kernel
    ("bf16", 64, 30, 424, O.I8, True, False),        # padded to 448: 9 rows a wave
    ("f32", 1, 29, 576, O.I8, False, False),
    ("bf16", 256, 23, 768, O.E4M3, True, True),      # 5 rows a wave
    ("bf16", 256, 5, 768, O.F64, False, False),      # the rotated values themselves
    ("bf16", 64, 21, 960, O.I8, True, False),        # 4 rows a wave, 15 lanes each
    ("f32", 64, 13, 1088, O.I8, True, False),        # 3 rows a wave
    ("bf16", 512, 7, 1536, O.E5M2, False, True),     # 2 rows a wave
    ("bf16", 64, 9, 1984, O.I8, True, False),
    ("bf16", 64, 6, 2112, O.I8, True, True),         # a row a wave, 33 lanes
    ("f32", 256, 5, 2304, O.E4M3, False, False),
    ("bf16", 512, 5, 3584, O.I8, True, False),
    ("f32", 64, 6, 4032, O.F64, True, False),
]


@pytest.mark.parametrize("io,block,rows,cols,qt,signs,sr", CASES)
def test_rows_that_do_not_divide_a_wave(io, block, rows, cols, qt, signs, sr):
    rng = np.random.default_rng(rows * 11 + cols + block)
    x = synth.activations(rng, rows, cols)
    if io == "bf16":
        x = synth.bf16_bits(x)
    words = synth.sign_words(O.padded_len(cols, block), seed=cols) if signs else None
    q, s = H.fwht_quant(to_dev(x), axis=H.ROWS, block=block, q_dtype=Q_TORCH[qt],
                        signs=signs_dev(words) if signs else None,
                        rounding="stochastic" if sr else "nearest", seed=SEED64, counter=COUNTER64)
    torch.cuda.synchronize()
    want, ws = O.fwht_quant(x, O.ROWS, block, qt, precision=32, signs=words,
                            rounding=O.STOCHASTIC if sr else O.RNE, key=KEY, ctr_hi=CTR)
    assert np.array_equal(codes_to_np(q), want)
    assert np.array_equal(s.cpu().numpy().astype(np.float64), ws)


def _long_call(rows, cols, block):
    """Zeros but for the last rows: their codes and scales, those of a call on them alone, and the
    first places where a row before them has a code or a scale that is not 0."""
    tail = 96
    g = torch.Generator(device=DEV)
    g.manual_seed(rows % 1000)
    x = torch.zeros((rows, cols), dtype=BF16, device=DEV)
    x[-tail:] = torch.randn((tail, cols), generator=g, device=DEV).to(BF16)
    q = torch.empty((rows, H.padded_len(cols, block)), dtype=torch.int8, device=DEV)
    for at in range(0, rows, 1 << 22):  # pieces: an index of one fill passes 32 bits
        q[at:at + (1 << 22)].fill_(1)
    s = torch.full((rows,), 7.0, device=DEV)
    H.fwht_quant(x, H.ROWS, block, q=q, scale=s)
    want = H.fwht_quant(x[-tail:].contiguous(), H.ROWS, block)
    assert torch.equal(q[-tail:], want[0]) and torch.equal(s[-tail:], want[1])
    assert not s[:-tail].any()
    for at in range(0, rows - tail, 1 << 22):
        assert not q[at:min(at + (1 << 22), rows - tail)].any()


def test_more_short_rows_than_a_launch_has_threads():
    # a workgroup of 64 threads a row would be 2^32 threads, which a launch drops without an error
    _long_call(2 ** 26 + 5, 192, 64)


def test_more_rows_than_a_launch_has_threads():
    rows = 2 ** 25 + 5  # of 4096 codes each, 64 threads a row: two launches
    if torch.cuda.mem_get_info()[0] < 150 * 2 ** 30:
        pytest.skip("137 GB of codes")
    _long_call(rows, 8, 4096)


@pytest.mark.parametrize("cols,block", [(320, 64), (1088, 16), (3136, 64)])
def test_large_fp32_calls_have_the_bits_of_small_ones(cols, block):
    # past 2^25 elements such rows take another kernel
    rows = 2 ** 25 // cols + 40
    g = torch.Generator(device=DEV)
    g.manual_seed(cols)
    x = torch.randn((rows, cols), generator=g, device=DEV)
    signs = H.hadamard_signs(cols, 3, DEV)
    for kw in ({}, dict(signs=signs, q_dtype=torch.float8_e4m3fn)):
        q, s = H.fwht_quant(x, H.ROWS, block, **kw)
        for at in (0, rows // 2):
            part = x[at:at + rows // 2]
            want = H.fwht_quant(part, H.ROWS, block, **kw)
            assert torch.equal(q[at:at + rows // 2].view(torch.uint8), want[0].view(torch.uint8))
            assert torch.equal(s[at:at + rows // 2], want[1])

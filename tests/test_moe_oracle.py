"""Pins of the oracle of routing, grouped products and block-scaled E4M3: values by hand, and properties that a
wrong one breaks."""
import numpy as np
import torch

import oracle
from oracle import moe

INF = np.inf


def test_choice_by_hand():
    l = np.array([[1.0, 3.0, 3.0, -INF], [-INF, np.nan, -INF, -INF], [INF, 0.0, -0.0, INF], [0.0, -0.0, np.nan, -5.0]])
    ids, w = moe.choose(l, 2, True)
    assert ids.tolist() == [[1, 2], [-1, -1], [0, 3], [0, 1]]
    assert w.tolist() == [[0.5, 0.5], [0.0, 0.0], [0.5, 0.5], [0.5, 0.5]]
    ids, w = moe.choose(l, 3, False)
    assert ids.tolist() == [[1, 2, 0], [-1, -1, -1], [0, 3, 1], [0, 1, 3]]
    assert np.allclose(w[0], np.exp([0, 0, -2]) / (2 + np.exp(-2))) and w[2].tolist() == [0.5, 0.5, 0.0]


def test_plan_by_hand():
    offsets, rows, places = moe.plan([[2, 0], [0, -1], [2, 3]], 4)
    assert offsets.tolist() == [0, 2, 2, 4, 5]
    assert rows.tolist() == [1, 2, 0, 4, 5, -1]
    assert places.tolist() == [2, 0, 1, -1, 3, 4]


def test_combine_by_hand():
    out, size = moe.combine(np.array([[1.0], [10.0]]), np.array([[0.5, -2.0], [3.0, 4.0]]), [1, 0, -1, 1])
    assert out.tolist() == [[3.0], [40.0]] and size.tolist() == [[7.0], [40.0]]


def test_dequant_agrees_with_the_dense_oracle():
    rng = np.random.default_rng(0)
    q = torch.from_numpy(rng.integers(-2 ** 31, 2 ** 31, (64, 3), dtype=np.int64).astype(np.int32))
    z = torch.from_numpy(rng.integers(-2 ** 31, 2 ** 31, (2, 3), dtype=np.int64).astype(np.int32))
    s = torch.rand(2, 24, dtype=torch.float32).half()
    for zeros in (z, None):
        w = moe.dequant(q.numpy(), s.double().numpy(), None if zeros is None else zeros.numpy(), 32)
        want = oracle.get().w4a16(torch.eye(64).half(), q, s, zeros, 32)
        assert np.array_equal(w, want)


def test_codes():
    assert moe.E4M3[1] == 2.0 ** -9 and moe.E4M3[8] == 2.0 ** -6 and moe.E4M3[126] == 448 and moe.E4M3[0x38] == 1
    every = np.array([c for c in range(256) if c & 127 != 127], dtype=np.uint8)
    assert np.array_equal(moe.encode(moe.decode(every)), every)
    t = torch.from_numpy(every).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(t, moe.decode(every))
    v = torch.randn(20000, generator=torch.Generator().manual_seed(0)) * 20
    v = torch.cat((v, torch.tensor([17.0, 19.0, 2.0 ** -10, 3 * 2.0 ** -10, -0.0])))  # ties, and half the smallest
    assert np.array_equal(moe.encode(v.numpy()), v.to(torch.float8_e4m3fn).view(torch.uint8).numpy())


def test_block_quant_by_hand():
    x = np.zeros((2, 160))
    x[0, 3], x[0, 130], x[1, 159] = 448.0, -1.0, 2.0 ** -24
    codes, s = moe.block_quant(x)
    assert s.shape == (2, 2) and s[0, 0] == 1 and s[0, 1] == np.float32(1 / 448) and s[1, 0] == 0
    assert codes[0, 3] == 126 and codes[0, 130] == 254 and codes[1, 159] == 126 and (codes != 0).sum() == 3
    assert np.array_equal(moe.block_values(codes, s, 1)[0, [3, 130]], [448.0, -448 * float(np.float32(1 / 448))])

"""Pins of the paged-cache oracle on the CPU: against torch's softmax, and its page state against
counting."""
import numpy as np
import torch

from oracle import cache as OC
from tests import cache_util as U


def test_attend_is_softmax():
    rng = np.random.default_rng(1)
    q, k, v = rng.standard_normal((5, 4, 16)), rng.standard_normal((30, 2, 16)), rng.standard_normal((30, 2, 16))
    see = OC.window_rows(5, 30, 7, 2)
    out, lse, mag, big, seen = OC.attend(q, k, v, see, 0.3)
    for h in range(4):
        x = torch.from_numpy(0.3 * q[:, h] @ k[:, h // 2].T).masked_fill(torch.from_numpy(~see), -torch.inf)
        assert np.allclose(out[:, h], (torch.softmax(x, 1) @ torch.from_numpy(v[:, h // 2])).numpy(), atol=1e-12)
        assert np.allclose(lse[:, h], torch.logsumexp(x, 1).numpy(), atol=1e-12)
    assert seen.tolist() == [9] * 5 and np.all(mag >= np.abs(out) - 1e-15) and np.all(big > 0)


def test_masks():
    see = OC.window_rows(3, 6, 2, 1)
    assert see.astype(int).tolist() == [[1, 0, 1, 1, 0, 0], [1, 0, 0, 1, 1, 0], [1, 0, 0, 0, 1, 1]]
    chain = np.tril(np.ones((3, 3), bool))
    assert np.array_equal(OC.tree_rows(chain, 6, 4, 0)[:, :3], OC.window_rows(3, 6, 4, 0)[:, :3])
    none = np.zeros((2, 2), bool)
    assert OC.tree_rows(none, 5, 2, 0).astype(int).tolist() == [[0, 1, 1, 0, 0]] * 2


def test_packing_round_trips():
    rng = np.random.default_rng(2)
    bits = U.tree_bits(rng, 70)
    w = U.pack_bits(bits, 2).numpy().view(np.uint64)
    for i in range(70):
        assert [bool(w[i, j // 64] >> np.uint64(j % 64) & np.uint64(1)) for j in range(70)] == bits[i].tolist()
    x = torch.randn(4, 128)
    assert torch.allclose(U.unpack_fp8(U.pack_fp8(x)), x.double(), rtol=2 ** -4, atol=1e-2)


def test_rotation_keeps_lengths_and_angles():
    x = np.random.default_rng(3).standard_normal((2, 1, 8))
    y = OC.qk_norm_rope(x, None, 0, [0, 5], [1.0, 0.1], 4, False)
    assert np.array_equal(y[0], x[0]) and np.array_equal(y[..., :4], x[..., :4])
    z = (x[1, 0, 4] + 1j * x[1, 0, 5]) * np.exp(5j)
    assert np.allclose([y[1, 0, 4], y[1, 0, 5]], [z.real, z.imag])
    h = OC.qk_norm_rope(x, None, 0, [0, 5], [1.0, 0.1], 4, True)
    z = (x[1, 0, 5] + 1j * x[1, 0, 7]) * np.exp(0.5j)
    assert np.allclose([h[1, 0, 5], h[1, 0, 7]], [z.real, z.imag])
    n = OC.qk_norm_rope(np.full((1, 1, 8), 3.0), np.arange(8), 0, [0], [], 0, False)
    assert np.allclose(n[0, 0], np.arange(8))


def test_pages_by_hand():
    p = OC.Pages([np.arange(8, dtype=np.uint8).reshape(8, 1, 1, 1).repeat(64, 2)], np.full((3, 4), -1, np.int32),
                 np.zeros(3, np.int32), np.zeros(8, np.int32), np.arange(8, dtype=np.int32), 8)
    assert p.grow([0, 1], [130, 10]) == [1, 1]
    assert p.table[0].tolist() == [7, 6, 5, -1] and p.table[1, 0] == 4 and p.n_free == 4
    assert p.fork([0], [2], False) == [1]
    assert p.table[2].tolist() == [7, 6, 3, -1] and p.ref.tolist() == [0, 0, 0, 1, 1, 1, 2, 2]
    assert p.pools[0][3].max() == 5
    assert p.compact([0], [128], [[129]], [1]) == [1] and p.lens[0] == 129
    assert p.compact([0], [0], [[1]], [1]) == [0]                        # shared
    assert p.free_requests([0, 2]) == [1, 1] and p.n_free == 7 and p.free[:7].tolist() == [0, 1, 2, 3, 5, 6, 7]

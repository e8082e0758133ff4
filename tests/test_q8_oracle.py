"""The 8-bit cache's oracle: pinned by closed forms and by PyTorch's own float8 type."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from oracle import q8_oracle as Q  # noqa: E402


def test_code_values_are_float8_e4m3fn():
    t = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(t, Q.CODE, equal_nan=True)


def test_codes_round_to_nearest_even():
    r = np.random.default_rng(0)
    x = np.concatenate([r.uniform(-448, 448, 20000), r.standard_normal(20000) * 0.02, Q.CODE[:127],
                        (Q.CODE[:126] + Q.CODE[1:127]) / 2, [0.0, -0.0]])
    c = Q.codes(x[None], np.zeros(1, int))[0]
    t = torch.as_tensor(x).float().to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    same = x == x.astype(np.float32)                 # fp32 holds it, so the cast rounds once
    assert np.array_equal(c[same], t[same])
    assert np.array_equal(Q.codes(np.array([[np.nan, np.inf, -np.inf]]), np.zeros(1, int))[0], [0x7F] * 3)


def test_exponents():
    a = np.array([[0.0], [448.0], [448.5], [1.0], [1.75], [1.7501], [3e38], [1e-30], [np.inf], [np.nan]])
    assert Q.exponent(a).tolist() == [-56, 0, 1, -8, -8, -7, 120, -56, -56, -56]
    x = np.array([[5.0, np.inf, -900.0, np.nan]])
    assert Q.exponent(x).tolist() == [2]
    held = Q.values(Q.codes(x, Q.exponent(x)), Q.exponent(x) + 127)
    assert held[0, 0] == 5.0 and held[0, 2] == -896.0 and np.isnan(held[0, [1, 3]]).all()


def test_norm_and_rotation():
    r = np.random.default_rng(1)
    x = r.standard_normal((5, 3, 64))
    y = Q.norm(x, np.ones(64), 0.0)
    assert np.allclose((y * y).mean(-1), 1.0)
    z, _ = Q.rope(x, [0, 1, 7, 100000, -3], 1e4)
    assert np.allclose(z[0], x[0]) and np.allclose(np.linalg.norm(z, axis=-1), np.linalg.norm(x, axis=-1))
    c, s = np.cos(1.0), np.sin(1.0)
    assert np.allclose(z[1, :, 0], x[1, :, 0] * c - x[1, :, 32] * s)
    a, b = Q.rope(x[:1], [11], 1e4)[0], Q.rope(x[:1], [4], 1e4)[0]        # relative positions
    a2, b2 = Q.rope(x[:1], [17], 1e4)[0], Q.rope(x[:1], [10], 1e4)[0]
    assert np.allclose((a[0, 0] * b[0, 1]).sum(), (a2[0, 0] * b2[0, 1]).sum())


def test_attention_is_pytorch_s():
    r = np.random.default_rng(2)
    n, L, hq, hkv, D = 4, 19, 6, 2, 8
    q, k, v = r.standard_normal((n, hq, D)), r.standard_normal((L, hkv, D)), r.standard_normal((L, hkv, D))
    o, lse, _, _ = Q.attention(q, k, v, n, 0.3)
    t = lambda a: torch.as_tensor(a).transpose(0, 1)  # noqa: E731
    mask = torch.ones(n, L, dtype=torch.bool).tril(L - n)
    kk, vv = t(k).repeat_interleave(3, 0), t(v).repeat_interleave(3, 0)
    ref = torch.nn.functional.scaled_dot_product_attention(t(q), kk, vv, attn_mask=mask, scale=0.3)
    assert np.allclose(o, ref.transpose(0, 1).numpy())
    z = (0.3 * t(q) @ kk.transpose(1, 2)).masked_fill(~mask, -np.inf)
    assert np.allclose(lse.T, torch.logsumexp(z, -1).numpy())
    assert np.allclose(Q.attention(np.zeros_like(q), k, v, n, 1.0)[0][3, 0], v[:, 0].mean(0))


def test_hidden_rows_are_not_seen():
    r = np.random.default_rng(3)
    q, k, v = r.standard_normal((1, 1, 8)), r.standard_normal((6, 1, 8)), r.standard_normal((6, 1, 8))
    o, _, _, _ = Q.attention(q, k[[0, 2, 5]], v[[0, 2, 5]], 1, 1.0)
    k[[1, 3, 4]] = np.nan
    assert np.allclose(Q.attention(q, k, v, 1, 1.0)[0], o)
    k[:] = np.nan
    o, lse, _, _ = Q.attention(q, k, v, 1, 1.0)
    assert (o == 0).all() and np.isneginf(lse).all()

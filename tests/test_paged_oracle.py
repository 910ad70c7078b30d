"""The paged-cache oracle pinned on the CPU: the code table and the encoder against torch's
float8_e4m3fn, the scale against its definition, and chunk attention against the decode
oracle and the causal attention oracle."""
import numpy as np
import pytest
import torch

from oracle import attention_oracle as A
from oracle import decode_oracle as D
from oracle import paged_oracle as P
from tests.paged_inputs import Batch


def test_code_values_are_e4m3():
    codes = torch.arange(256, dtype=torch.int32).to(torch.uint8)
    want = codes.view(torch.float8_e4m3fn).float().double().numpy()
    assert np.array_equal(P.e4m3_values(), want, equal_nan=True)


def test_encode_rounds_like_e4m3_and_scales_by_powers_of_two():
    g = torch.Generator("cpu").manual_seed(1)
    x = (torch.randn(200, 64, generator=g) * torch.exp2(torch.randint(-30, 30, (200, 1), generator=g))
         ).to(torch.bfloat16).double()
    codes, ex = P.encode(x.numpy())
    e = ex.astype(np.int64) - 127
    amax = x.abs().amax(-1).numpy()
    assert (amax <= 448.0 * 2.0 ** e).all() and (amax > 448.0 * 2.0 ** (e - 1)).all()
    y = (x / torch.exp2(torch.from_numpy(e).double())[:, None]).float().to(torch.float8_e4m3fn)
    assert np.array_equal(codes, y.view(torch.uint8).numpy())
    # the value of every code is exact in bf16
    back = P.decode(codes, ex)
    assert np.array_equal(back, torch.from_numpy(back).to(torch.bfloat16).double().numpy())


def test_encode_special_rows():
    x = np.zeros((4, 8))
    x[1, 3] = 448.0
    x[2, :3] = [448.5, np.inf, np.nan]
    x[3, 0] = 2.0 ** -133
    codes, ex = P.encode(x)
    assert ex.tolist() == [0, 127, 128, 0]
    assert codes[1, 3] == 126 and codes[2, 1] == 127 and codes[2, 2] == 127
    assert P.decode(codes, ex)[2, 0] == 448.0        # 224.25 rounds to 224, under 2^1
    assert P.decode(codes, ex)[3, 0] == 2.0 ** -133


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_chunks_of_equal_length_are_decode(kind):
    w = Batch([3, 3, 3], [3, 20, 57], kind=kind, seed=2)
    kc, vc = w.k_cache, w.v_cache
    if kind == "e4m3":
        kc = torch.from_numpy(P.decode(kc.numpy(), w.kv_exp[..., 0].numpy()))
        vc = torch.from_numpy(P.decode(vc.numpy(), w.kv_exp[..., 1].numpy()))
    for mask, window, score in ((0, 0, 0), (1, 0, A.SCORE_ALIBI), (2, 9, A.SCORE_SOFTCAP)):
        o, z, _ = P.chunk_forward(w.q, w.k_cache, w.v_cache, w.kv_exp, w.table, w.offsets, w.lens,
                                  0.125, mask, window, score, 7.0)
        qd = w.q.reshape(3, 3, w.Hq, w.d).transpose(1, 2)
        od, zd = D.decode_forward(qd, kc, vc, w.table, w.lens, 0.125, mask, window, score, 7.0)
        np.testing.assert_allclose(o.reshape(3, 3, w.Hq, w.d).transpose(0, 2, 1, 3), od, rtol=1e-12, atol=1e-12)
        np.testing.assert_allclose(z.reshape(3, 3, w.Hq).transpose(0, 2, 1), zd, rtol=1e-12, atol=1e-12)


def test_whole_prompts_are_causal_attention():
    w = Batch([5, 0, 33], [5, 7, 33], page=8, seed=3)
    o, z, _ = P.chunk_forward(w.q, w.k_cache, w.v_cache, None, w.table, w.offsets, w.lens, 0.2, 1)
    for b in (0, 2):
        t0, t1 = w.offsets[b], w.offsets[b + 1]
        K, V = P.sequence(w.k_cache, w.v_cache, None, w.table[b], 0, w.lens[b])
        bh = lambda x: np.asarray(x, dtype=np.float64).transpose(1, 0, 2)[None]  # noqa: E731
        o_ref, z_ref = A.forward(bh(w.q[t0:t1].double()), bh(K), bh(V), 0.2, mask_kind=A.MASK_CAUSAL)
        np.testing.assert_allclose(o[t0:t1].transpose(1, 0, 2), o_ref[0], rtol=1e-12, atol=1e-12)
        np.testing.assert_allclose(z[t0:t1].T, z_ref[0], rtol=1e-12, atol=1e-12)


def test_written_tokens_read_back():
    w = Batch([2, 4], [20, 4], kind="e4m3", seed=4)
    kc, vc, ex = w.written()
    K, V = P.sequence(kc.numpy(), vc.numpy(), ex.numpy(), w.table[0], 18, 20)
    for got, x in ((K, w.k[:2]), (V, w.v[:2])):
        # e4m3 keeps 4 significant bits: half a step is 2^-4 of the value, 2^-10 of the scale
        x = x.double().numpy()
        top = np.abs(x).max(axis=-1, keepdims=True)
        assert (np.abs(got - x) <= np.maximum(2.0 ** -4 * np.abs(x), 2.0 ** -10 * top / 224)).all()

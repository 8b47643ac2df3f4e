"""Tensors of another type or size than a call reads are refused before any pointer is taken."""
import pytest
import torch

import qk_normed_latent_gb300 as Q

N, S, B, H, G, D_C, D_H, D_R = 5, 64, 2, 16, 4, 256, 64, 32
F32, BF16, I32, I64, U8 = torch.float32, torch.bfloat16, torch.int32, torch.int64, torch.uint8


def zeros(*shape, dtype=F32):
    return torch.zeros(shape, dtype=dtype)


def append(**kw):
    a = dict(c_new=zeros(N, D_C), k_rope_new=zeros(N, D_R), w_k=zeros(G, D_C, D_H), gamma_rope_k=zeros(D_R),
             slot_mapping=zeros(N, dtype=I64), kv_cache=zeros(S, D_C + 2 * D_R, dtype=U8), kv_scale=zeros(S),
             ak_cache=zeros(S, G), eps=1e-6, positions=zeros(N, dtype=I32), rope_theta=1e4)
    a.update(kw)
    return Q.prepare_append_q8(**a)


@pytest.mark.parametrize("name,t", [
    ("c_new", zeros(N, D_C, dtype=BF16)), ("c_new", zeros(N, D_C, dtype=torch.float64)),
    ("k_rope_new", zeros(N, D_R, dtype=BF16)), ("k_rope_new", zeros(N - 1, D_R)),
    ("w_k", zeros(G, D_C, D_H, dtype=BF16)), ("w_k", zeros(G, D_C // 2, D_H)),
    ("gamma_rope_k", zeros(D_R - 1)), ("gamma_rope_k", zeros(D_R, dtype=BF16)),
    ("slot_mapping", zeros(N, dtype=I32)), ("slot_mapping", zeros(N - 1, dtype=I64)), ("slot_mapping", None),
    ("ak_cache", zeros(S - 1, G)), ("ak_cache", zeros(S, G, dtype=BF16)),
    ("positions", zeros(N, dtype=I64)), ("positions", zeros(N - 1, dtype=I32)),
])
def test_append_q8(name, t):
    with pytest.raises(ValueError, match=name):
        append(**{name: t})


def decode(**kw):
    a = dict(q_tilde=zeros(B, 1, H, D_C, dtype=BF16), alpha_q=zeros(B, 1, H), q_rope=zeros(B, 1, H, D_R),
             gamma_rope_q=zeros(D_R), kv_cache=zeros(S, D_C + 2 * D_R, dtype=U8), ak_cache=zeros(S, G),
             seq_lens=zeros(B, dtype=I32), page_table=zeros(B, 3, dtype=I32), page_size=16, max_pages=3, G=G,
             softmax_scale=0.1, eps=1e-6, o=zeros(B, 1, H, D_C), lse=zeros(B, 1, H), kv_scale=zeros(S))
    a.update(kw)
    return Q.prepare_decode(**a)


@pytest.mark.parametrize("name,t", [
    ("alpha_q", zeros(B, 1, H - 1)), ("alpha_q", zeros(B, 1, H, dtype=BF16)), ("alpha_q", None),
    ("q_rope", zeros(B, 1, H, D_R, dtype=BF16)), ("q_rope", zeros(B, 1, 1, D_R)), ("gamma_rope_q", zeros(D_R // 2)),
    ("ak_cache", zeros(S, G - 1)), ("ak_cache", None), ("seq_lens", zeros(B, dtype=I64)),
    ("seq_lens", zeros(B - 1, dtype=I32)), ("page_table", zeros(B, 2, dtype=I32)), ("page_table", zeros(B, 3, dtype=I64)),
    ("o", zeros(B, 1, H, D_C // 2)), ("o", zeros(B, 1, H, D_C, dtype=torch.float16)), ("lse", zeros(B, 1, 1)),
    ("q_tilde", zeros(B, 1, H, D_C)),
])
def test_decode(name, t):
    with pytest.raises(ValueError, match=name):
        decode(**{name: t})


@pytest.mark.parametrize("name,kw", [
    ("kv_cache", dict(kv_cache=zeros(S, D_C, dtype=BF16))), ("q_tilde", dict(q_tilde=zeros(B, 1, H, D_C))),
])
def test_windowed_decode_of_a_bf16_cache(name, kw):
    with pytest.raises(ValueError, match=name):
        decode(**{"kv_cache": zeros(S, D_C + D_R, dtype=BF16), "kv_scale": None, "window": 9, **kw})


def test_right_ones_pass_the_checks():
    """Everything but the device: the last check before a pointer is taken."""
    with pytest.raises(ValueError, match="CUDA device"):
        append()
    with pytest.raises(ValueError, match="CUDA device"):
        decode()

"""CPU side of the serving operators' edges: byte counts of a step, and what four e4m3 parts hold
of a bf16 query value."""
import torch

from io_aware_exact_26_b200 import accounting as acc


def test_serving_step_bytes():
    T, Hq, Hkv, d, cached = 3, 8, 2, 64, 1000
    new = T * (Hq + 2 * Hkv) * d * 2                       # q, k, v of the new tokens in
    put = T * Hq * d * 2 + 2 * T * Hkv * d * 2             # q rotated out, k and v into a bf16 cache
    attend = T * Hq * d * 2 + 2 * cached * Hkv * d * 2 + T * Hq * d * 2 + T * Hq * 4
    assert acc.min_bytes_serve(T, Hq, Hkv, d, cached, 2 * d) == new + put + attend
    # a row of an e4m3 cache: d codes and a scale byte
    less = 2 * (T + cached) * Hkv * (2 * d - (d + 1))
    assert acc.min_bytes_serve(T, Hq, Hkv, d, cached, d + 1) == new + put + attend - less
    # bound by the cache: one token on a long context costs what decoding over the dense cache does
    dense = acc.min_bytes_decode(16, 32, 8, 1, 32768, 128)
    assert 0 <= acc.min_bytes_serve(16, 32, 8, 128, 16 * 32768, 256) - dense < 1e-3 * dense


def test_four_e4m3_parts_of_a_query_value():
    """Every positive bf16 value as a query row's element, its row's largest magnitude between 224 and
    448 in the units of the split: exact down to 2^-35 of that magnitude, within 2^-43 of it below."""
    bits = torch.arange(1, 0x7f80, dtype=torch.int32).to(torch.int16)
    v = bits.view(torch.bfloat16).double()
    v = v[v <= 448]
    rest, total, unit = v.clone(), torch.zeros_like(v), 1.0
    for step in (16.0, 2.0 ** 18, 16.0, 1.0):
        assert float(rest.abs().max()) <= 448
        part = rest.float().to(torch.float8_e4m3fn).double()
        total += part * unit
        rest = (rest - part) * step
        unit /= step
    err = (total - v).abs()
    for top in (224.0, 448.0):
        assert bool((err[v >= 2.0 ** -35 * top] == 0).all()) and float(err.max()) <= 2.0 ** -43 * top

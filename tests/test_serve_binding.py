"""What the binding of the serving calls takes for a tensor (no GPU needed)."""
import numpy as np
import pytest
import torch

import hybrid_attention_ssm_hymba_b200 as H

P = 1 << 20   # an aligned address that nothing may read


@pytest.mark.parametrize("thing", [b"0123456789abcdef", "0123456789abcdef", bytearray(16), np.zeros(4), [1, 2], 1.0])
def test_only_tensors_and_addresses_are_pointers(thing):
    """bytes and str would pass as pointers to host memory, which a kernel would read."""
    with pytest.raises(AttributeError):
        H.hymba_rmsnorm(thing, P, 1, 16, 1e-5, H.HYMBA_BF16, stream=0)
    with pytest.raises(AttributeError):
        H.hymba_quantize_w4(P, thing, P, 16, 128, 64, H.HYMBA_BF16, stream=0)
    with pytest.raises(AttributeError):
        H.hymba_workspace_status(thing, stream=0)


def _pool(cache=torch.bfloat16, **kw):
    a = dict(pages=torch.zeros(2, 6, 16, 2, 32, dtype=cache), page_table=torch.zeros(3, 4, dtype=torch.int32), page_size=16,
             n_kv_heads=2, head_dim=32, cache_type=H.HYMBA_CACHE_BF16)
    a.update(kw)
    return a


def test_paged_kv_of_dense_tensors():
    kv = H.make_paged_kv(**_pool())
    assert (kv.n_pages, kv.table_ld, kv.scales) == (6, 4, None)
    kv = H.make_paged_kv(**_pool(torch.float8_e4m3fn, cache_type=H.HYMBA_CACHE_E4M3, scales=torch.zeros(2, 6, 2, 16)))
    assert kv.n_pages == 6 and kv.scales
    assert H.make_paged_kv(**_pool(pages=torch.zeros(2 * 6 * 16, 64, dtype=torch.bfloat16))).n_pages == 6
    H.make_paged_kv(**_pool(scales=torch.zeros(1)))   # (a cache that has no scales does not look at them)
    assert H.make_paged_kv(**_pool(page_table=torch.zeros(3, 9, dtype=torch.int32)[1:])).table_ld == 9   # rows of a table


@pytest.mark.parametrize("bad", [
    dict(page_table=torch.zeros(3, 9, dtype=torch.int32)[:, :4]),                # its rows are 9 apart, not 4
    dict(page_table=torch.zeros(4, 3, dtype=torch.int32).t()), dict(page_table=torch.zeros(3, 4, dtype=torch.int64)),
    dict(page_table=torch.zeros(3, 4)), dict(pages=torch.zeros(2, 6, 16, 2, 64, dtype=torch.bfloat16)[..., :32]),
    dict(pages=torch.zeros(6, 2, 16, 2, 32, dtype=torch.bfloat16).transpose(0, 1)),
    dict(pages=torch.zeros(2, 6, 16, 2, 32)), dict(pages=torch.zeros(2 * 6 * 16 * 64 + 8, dtype=torch.bfloat16)),
    dict(pages=torch.zeros(2, 6, 16, 2, 32, dtype=torch.uint8), cache_type=H.HYMBA_CACHE_E4M3,
         scales=torch.zeros(2, 6, 2, 32)[..., :16]),
    dict(pages=torch.zeros(2, 6, 16, 2, 32, dtype=torch.uint8), cache_type=H.HYMBA_CACHE_E4M3,
         scales=torch.zeros(2, 6, 2, 16, dtype=torch.bfloat16)),
    dict(pages=torch.zeros(2, 6, 16, 2, 32, dtype=torch.uint8), cache_type=H.HYMBA_CACHE_E4M3, scales=torch.zeros(2, 5, 2, 16)),
])
def test_paged_kv_refuses_what_it_would_misread(bad):
    """The descriptor's pitches come from the shapes: strided tensors, or elements of another size, would
    be read as other rows without an error."""
    with pytest.raises(ValueError):
        H.make_paged_kv(**_pool(**bad))


@pytest.mark.parametrize("dtype,cache", [(H.HYMBA_F32, H.HYMBA_CACHE_F32), (H.HYMBA_F32, H.HYMBA_CACHE_E4M3),
                                         (H.HYMBA_BF16, H.HYMBA_CACHE_BF16), (H.HYMBA_BF16, H.HYMBA_CACHE_E4M3)])
@pytest.mark.parametrize("hq,hkv,table_ld", [(16, 4, 512), (1, 1, 3), (48, 1, 40), (4, 4, 1), (64, 64, 2048)])
def test_a_workspace_for_the_largest_call_serves_smaller_ones(hq, hkv, table_ld, dtype, cache):
    """Sizes do not shrink as batch, rows or the longest chunk grow."""
    kv = H.hymba_paged_kv_t()
    for name, v in dict(pages=P, scales=P, page_table=P, n_pages=1000, page_size=64, table_ld=table_ld, n_kv_heads=hkv,
                        head_dim=128, cache_type=cache).items():
        setattr(kv, name, v)

    def size(batch, total, most):
        return H.hymba_paged_attention_workspace_size(kv, batch, total, most, hq, dtype)

    for sizes in ([size(8, total, 8) for total in range(0, 700)], [size(8, 700, most) for most in range(1, 700)],
                  [size(batch, 700, 8) for batch in range(1, 2000, 7)]):
        assert min(sizes) >= 256 and sizes == sorted(sizes)

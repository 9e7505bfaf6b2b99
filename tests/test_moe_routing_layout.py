"""A routing's fields share one allocation: attributes, dictionary, iteration and the addresses that the calls pass
come from one layout, and a copy of a routing is a routing."""
import copy
import pickle

import pytest
import torch

import moe_nvfp4_gemm_gb300 as m

SIZES = [(0, 1, 1), (1, 1, 1), (1, 256, 8), (7, 3, 2), (1001, 8, 2), (40, 1024, 32)]


def shape_of(t):
    return t.data_ptr(), tuple(t.shape), t.stride(), t.dtype


def fresh(T, E, k, device="cpu"):
    return m.MoeRouting(T, E, k, False, None, device, 12)


@pytest.mark.parametrize("T,E,k", SIZES)
def test_views_and_addresses_agree(T, E, k):
    shapes = {"topk_idx": (T, k), "topk_w": (T, k), "slot_row": (T, k), "counts": (E,), "expert_offsets": (E + 1,),
              "row_token": (T * k,), "mean_prob": (E,), "balance_loss": (1,), "routed_tokens": (1,)}
    a = fresh(T, E, k)
    one_by_one = {f: shape_of(getattr(a, f)) for f in reversed(m.MoeRouting._fields)}
    at_once = {f: shape_of(t) for f, t in a._asdict().items()}
    assert tuple(at_once) == m.MoeRouting._fields == tuple(m._routing_layout(T, E, k)[0])
    assert one_by_one == at_once and [shape_of(t) for t in a] == list(at_once.values())
    *fields, workspace = a._addresses()
    end = a._buf.data_ptr()
    for f, address in zip(m.MoeRouting._fields, fields):
        t = getattr(a, f)
        assert tuple(t.shape) == shapes[f] and t.is_contiguous()
        assert t.dtype == (torch.float32 if f in ("topk_w", "mean_prob", "balance_loss") else torch.int32)
        assert address == end
        if t.numel():
            assert t.data_ptr() == address
        end += 4 * t.numel()  # one behind the other, none over another
    assert end <= workspace < end + 16 and (workspace - a._buf.data_ptr()) % 16 == 0
    assert workspace + 48 == a._buf.data_ptr() + 4 * a._buf.numel()
    b = fresh(T, E, k)  # the other order: all at once, then the attributes
    assert [shape_of(t) for t in b] == [shape_of(getattr(b, f)) for f in m.MoeRouting._fields]
    assert all(x is y for x, y in zip(b, b))


@pytest.mark.parametrize("touched", [False, True])
@pytest.mark.parametrize("how", [copy.deepcopy, lambda r: pickle.loads(pickle.dumps(r))])
def test_a_copy_has_its_own_addresses(touched, how):
    r = fresh(5, 4, 2)
    r._buf.copy_(torch.arange(r._buf.numel()))
    if touched:
        r._asdict()
    c = how(r)
    assert (c.T, c.E, c.k) == (5, 4, 2) and c._buf.data_ptr() != r._buf.data_ptr()
    *fields, _ = c._addresses()
    for f, address, t in zip(m.MoeRouting._fields, fields, c):
        assert t.data_ptr() == address == getattr(c, f).data_ptr()
        assert torch.equal(t, getattr(r, f))


def test_unknown_attribute():
    with pytest.raises(AttributeError):
        fresh(1, 2, 1).weights


@pytest.mark.gpu
def test_gradient_from_a_copy():
    logits = torch.randn(300, 16, device="cuda")
    r = m.nvfp4_moe_route(logits, 2, renormalize=True)
    dw = torch.randn(300, 2, device="cuda")
    want = m.nvfp4_moe_route_backward(logits, r, d_w=dw, d_loss=torch.ones(1, device="cuda"))
    c = copy.deepcopy(r)
    r._buf.zero_()  # the copy does not lean on the first one's memory
    assert torch.equal(want, m.nvfp4_moe_route_backward(logits, c, d_w=dw, d_loss=torch.ones(1, device="cuda")))
